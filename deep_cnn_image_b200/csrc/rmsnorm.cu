// rmsnorm.cu -- root-mean-square norm of rows with the residual's addition,
// its gradient, and the conversion between bf16 and 8-bit rows.  All of it is
// bound by the bytes of its rows.
#include <cuda_bf16.h>

#include "f8.cuh"
#include "ff.h"
#include "kernels.h"
#include "ptx.cuh"

namespace alx {

namespace {

// Sum over the G threads (32 or a whole block of G) that share a row; the
// order is fixed, so results are reproducible.  `red` holds G / 32 floats.
template <int G>
__device__ __forceinline__ float row_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (G > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    v = lane < G / 32 ? red[lane] : 0.f;
#pragma unroll
    for (int o = G / 64; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    v = __shfl_sync(0xFFFFFFFFu, v, 0);
  }
  return v;
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x;
  f[1] = a.y;
  f[2] = a.z;
  f[3] = a.w;
  f[4] = b.x;
  f[5] = b.y;
  f[6] = b.z;
  f[7] = b.w;
}

// Largest finite magnitude of f over the 16 lanes that hold a block's 128
// values; f's infinities become NaN.
__device__ __forceinline__ float block_amax(float (&f)[8], uint32_t mask) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[i] = f8_finite(f[i]);
    a = fmaxf(a, fabsf(f[i]));
  }
#pragma unroll
  for (int o = 8; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(mask, a, o));
  return a;
}

__device__ __forceinline__ uint2 codes8(const float (&f)[8], float inv, int e5m2) {
  return make_uint2(f8_pack4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv, e5m2),
                    f8_pack4(f[4] * inv, f[5] * inv, f[6] * inv, f[7] * inv, e5m2));
}

// y = s * rstd * gamma with s = bf16(x + res), rstd = 1/sqrt(mean(s^2) + eps).
// One pass over the row: G threads hold it in registers as bf16 (NV vectors of
// 8 columns each, thread t the vectors t, t + G, ...), so the rounded s is
// also what the statistic and the gradient see.  16 neighbouring lanes hold
// one 128-column block of the 8-bit output.
template <int G, int NV>
__global__ void __launch_bounds__(G > 32 ? G : 256)
    k_rmsnorm_fwd(const bf16* x, const bf16* res,
                  const float* __restrict__ gamma, int64_t rows, int cols, float eps,
                  bf16* sum, bf16* y, float* rstd, uint8_t* q, uint8_t* scales) {
  __shared__ float red[32];
  grid_dep_launch();
  grid_dep_wait();
  const int t = G > 32 ? threadIdx.x : (threadIdx.x & 31);
  const int64_t row =
      G > 32 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;  // whole warps of a G = 32 block only
  const int nvec = cols >> 3;
  const bf16* xr = x + row * cols;
  uint4 v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)
    v[j] = t + j * G < nvec ? *reinterpret_cast<const uint4*>(xr + 8 * (t + j * G))
                            : make_uint4(0, 0, 0, 0);
  if (res) {
    uint4 r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j)
      r[j] = t + j * G < nvec
                 ? *reinterpret_cast<const uint4*>(res + row * cols + 8 * (t + j * G))
                 : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float a[8], b[8];
      unpack8_bits(v[j], a);
      unpack8_bits(r[j], b);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] += b[i];
      v[j] = pack8(a);
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float a[8];
    unpack8_bits(v[j], a);
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += a[i] * a[i];
  }
  ss = row_sum<G>(ss, red);
  const float r = 1.f / sqrtf(ss / static_cast<float>(cols) + eps);
  if (rstd && t == 0) rstd[row] = r;
  const int col_tiles = (cols + F8_TILE_COLS - 1) / F8_TILE_COLS;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int u = t + j * G;
    const bool live = u < nvec;
    if (live && sum) *reinterpret_cast<uint4*>(sum + row * cols + 8 * u) = v[j];
    if (!y && !q) continue;
    float a[8], g[8] = {};
    unpack8_bits(v[j], a);
    if (live) load8(gamma + 8 * u, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = a[i] * r * g[i];
    if (live && y) *reinterpret_cast<uint4*>(y + row * cols + 8 * u) = pack8(a);
    if (q) {
      if (!live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = 0.f;
      }
      const uint32_t s = f8_scale_byte(block_amax(a, 0xFFFFFFFFu), 0);
      if (live) {
        *reinterpret_cast<uint2*>(q + row * cols + 8 * u) = codes8(a, f8_scale_inv(s), 0);
        if ((u & 15) == 0) scales[f8_scale_at(row, u >> 4, col_tiles)] = static_cast<uint8_t>(s);
      }
    }
  }
}

// dx = rstd (t - s rstd^2 mean(t s)) + dsum, t = dy gamma.  A row is held in
// registers by G threads as above; a block (or warp) walks rows blockIdx.x,
// blockIdx.x + gridDim.x, ..., and a thread's columns are the same in all of
// them, so the sums of dy s rstd stay in registers and are written once per
// block, as one row of `parts`.
template <int G, int NV>
__global__ void __launch_bounds__(G > 32 ? G : 256)
    k_rmsnorm_bwd(const bf16* dy, const bf16* dsum, const bf16* __restrict__ sum,
                  const float* __restrict__ gamma, const float* __restrict__ rstd, int64_t rows,
                  int cols, bf16* dx, float* __restrict__ parts) {
  __shared__ float red[2][32];
  grid_dep_launch();
  grid_dep_wait();
  const int t = G > 32 ? threadIdx.x : (threadIdx.x & 31);
  const int64_t first =
      G > 32 ? blockIdx.x : static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t step = G > 32 ? gridDim.x : static_cast<int64_t>(gridDim.x) * 8;
  const int nvec = cols >> 3;
  float acc[NV][8] = {};
  int flip = 0;
  for (int64_t row = first; row < rows; row += step, flip ^= 1) {
    uint4 vd[NV], vs[NV];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = t + j * G;
      vd[j] = u < nvec ? *reinterpret_cast<const uint4*>(dy + row * cols + 8 * u) : zero;
      vs[j] = u < nvec ? *reinterpret_cast<const uint4*>(sum + row * cols + 8 * u) : zero;
    }
    const float r = rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = t + j * G;
      float d[8], s[8], g[8] = {};
      unpack8_bits(vd[j], d);
      unpack8_bits(vs[j], s);
      if (u < nvec) load8(gamma + 8 * u, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot += d[i] * g[i] * s[i];
        acc[j][i] += d[i] * (s[i] * r);
      }
    }
    dot = row_sum<G>(dot, red[flip]);
    const float c = r * r * (dot / static_cast<float>(cols));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int u = t + j * G;
      if (u < nvec) {
        float d[8], s[8], g[8], e[8] = {};
        unpack8_bits(vd[j], d);
        unpack8_bits(vs[j], s);
        load8(gamma + 8 * u, g);
        if (dsum) unpack8_bits(*reinterpret_cast<const uint4*>(dsum + row * cols + 8 * u), e);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = r * (d[i] * g[i] - s[i] * c) + e[i];
        *reinterpret_cast<uint4*>(dx + row * cols + 8 * u) = pack8(d);
      }
    }
  }
  if (!parts) return;
  float* p = parts + (G > 32 ? static_cast<size_t>(blockIdx.x) : static_cast<size_t>(first)) * cols;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int u = t + j * G;
    if (u < nvec) {
      *reinterpret_cast<float4*>(p + 8 * u) =
          make_float4(acc[j][0], acc[j][1], acc[j][2], acc[j][3]);
      *reinterpret_cast<float4*>(p + 8 * u + 4) =
          make_float4(acc[j][4], acc[j][5], acc[j][6], acc[j][7]);
    }
  }
}

// out[c] = sum over n rows of parts[.][c], in a fixed order: 32 columns per
// block, 16 groups of rows, then the groups.
__global__ void __launch_bounds__(512)
    k_sum_parts(const float* __restrict__ parts, int n, int cols, float* __restrict__ out) {
  __shared__ float red[16][33];
  grid_dep_launch();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (c < cols)
    for (int i = grp; i < n; i += 16) a += parts[static_cast<size_t>(i) * cols + c];
  red[grp][lane] = a;
  __syncthreads();
  if (grp == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 16; ++i) a += red[i][lane];
    out[c] = a;
  }
}

// 16 lanes per 128-column block, 8 values each.
__global__ void __launch_bounds__(256)
    k_f8_quant(const bf16* __restrict__ x, int64_t rows, int cols, int e5m2,
               uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  grid_dep_launch();
  grid_dep_wait();
  const int blocks = (cols + F8_BLOCK - 1) / F8_BLOCK;
  const int col_tiles = (cols + F8_TILE_COLS - 1) / F8_TILE_COLS;
  const int64_t total = rows * blocks;
  const int sub = threadIdx.x & 15;
  const uint32_t mask = 0xFFFFu << (threadIdx.x & 16);
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 16 + (threadIdx.x >> 4); b < total;
       b += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t row = b / blocks;
    const int blk = static_cast<int>(b - row * blocks);
    const int col = blk * F8_BLOCK + sub * 8;
    float f[8] = {};
    if (col < cols) unpack8_bits(*reinterpret_cast<const uint4*>(x + row * cols + col), f);
    const uint32_t s = f8_scale_byte(block_amax(f, mask), e5m2);
    if (col < cols)
      *reinterpret_cast<uint2*>(q + row * cols + col) = codes8(f, f8_scale_inv(s), e5m2);
    if (sub == 0) scales[f8_scale_at(row, blk, col_tiles)] = static_cast<uint8_t>(s);
  }
}

// 16 codes per thread.
__global__ void __launch_bounds__(256)
    k_f8_dequant(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scales, int64_t rows,
                 int cols, int e5m2, bf16* __restrict__ x) {
  grid_dep_launch();
  grid_dep_wait();
  const int vecs = cols >> 4;
  const int col_tiles = (cols + F8_TILE_COLS - 1) / F8_TILE_COLS;
  const int64_t total = rows * vecs;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = i / vecs;
    const int c = static_cast<int>(i - row * vecs);
    const uint4 w = *reinterpret_cast<const uint4*>(q + i * 16);
    const float sc = f8_scale_val(scales[f8_scale_at(row, c >> 3, col_tiles)]);
    uint32_t o[8];
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float v[4];
      f8_unpack4(in[k], e5m2, v);
      o[2 * k] = pack_bf16(v[0] * sc, v[1] * sc);
      o[2 * k + 1] = pack_bf16(v[2] * sc, v[3] * sc);
    }
    uint4* out = reinterpret_cast<uint4*>(x + i * 16);
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

int grid_for(int64_t blocks) {
  const int64_t most = static_cast<int64_t>(ff_num_sms()) * 16;
  return static_cast<int>(blocks < most ? blocks : most);
}

// Blocks of the backward: as many rows in flight as the SMs hold.
int bwd_grid(int64_t rows, int cols) {
  const int64_t want = cols <= 1024 ? (rows + 7) / 8 : rows;
  const int64_t most = static_cast<int64_t>(ff_num_sms()) * (cols <= 8192 ? 2 : 1);
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

int ff_num_sms() {
  static int cached[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!cached[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = n > 0 ? n : 148;
  }
  return cached[dev];
}

// Threads per row by its width: a warp up to 1024 columns (no block
// barrier, eight rows per block), 256 threads up to 16384, 1024 beyond.
#define ALX_ROWS(G_, NV_, KERNEL, GRID, ...) \
  e = ff_launch(KERNEL<G_, NV_>, GRID, G_ > 32 ? G_ : 256, 0, 0, s, __VA_ARGS__)
#define ALX_ROWS_BY_WIDTH(KERNEL, WARP_GRID, ROW_GRID, ...)                       \
  if (cols <= 256) ALX_ROWS(32, 1, KERNEL, WARP_GRID, __VA_ARGS__);               \
  else if (cols <= 512) ALX_ROWS(32, 2, KERNEL, WARP_GRID, __VA_ARGS__);          \
  else if (cols <= 1024) ALX_ROWS(32, 4, KERNEL, WARP_GRID, __VA_ARGS__);         \
  else if (cols <= 2048) ALX_ROWS(256, 1, KERNEL, ROW_GRID, __VA_ARGS__);         \
  else if (cols <= 4096) ALX_ROWS(256, 2, KERNEL, ROW_GRID, __VA_ARGS__);         \
  else if (cols <= 8192) ALX_ROWS(256, 4, KERNEL, ROW_GRID, __VA_ARGS__);         \
  else if (cols <= 16384) ALX_ROWS(256, 8, KERNEL, ROW_GRID, __VA_ARGS__);        \
  else if (cols <= 32768) ALX_ROWS(1024, 4, KERNEL, ROW_GRID, __VA_ARGS__);       \
  else ALX_ROWS(1024, 8, KERNEL, ROW_GRID, __VA_ARGS__)

cudaError_t launch_rmsnorm_fwd(const bf16* x, const bf16* res, const float* gamma, int64_t rows,
                               int cols, float eps, bf16* sum, bf16* y, float* rstd, uint8_t* q,
                               uint8_t* scales, cudaStream_t s) {
  const int64_t wg = (rows + 7) / 8, rg = rows;
  cudaError_t e = cudaSuccess;
  ALX_ROWS_BY_WIDTH(k_rmsnorm_fwd, wg, rg, x, res, gamma, rows, cols, eps, sum, y, rstd, q,
                    scales);
  count_launch();
  return e;
}

int rmsnorm_bwd_parts(int64_t rows, int cols) {
  return bwd_grid(rows, cols) * (cols <= 1024 ? 8 : 1);
}

cudaError_t launch_rmsnorm_bwd(const bf16* dy, const bf16* dsum, const bf16* sum,
                               const float* gamma, const float* rstd, int64_t rows, int cols,
                               bf16* dx, float* dgamma, float* parts, cudaStream_t s) {
  const int grid = bwd_grid(rows, cols);
  cudaError_t e = cudaSuccess;
  ALX_ROWS_BY_WIDTH(k_rmsnorm_bwd, grid, grid, dy, dsum, sum, gamma, rstd, rows, cols, dx,
                    dgamma ? parts : static_cast<float*>(nullptr));
  count_launch();
  if (dgamma && e == cudaSuccess) {
    e = ff_launch(k_sum_parts, (cols + 31) / 32, 512, 0, 0, s, parts,
                  rmsnorm_bwd_parts(rows, cols), cols, dgamma);
    count_launch();
  }
  return e;
}

cudaError_t launch_f8_quant(const bf16* x, int64_t rows, int cols, int e5m2, uint8_t* q,
                            uint8_t* scales, cudaStream_t s) {
  const int64_t blocks = rows * ((cols + F8_BLOCK - 1) / F8_BLOCK);
  count_launch();
  return ff_launch(k_f8_quant, grid_for((blocks + 15) / 16), 256, 0, 0, s, x, rows, cols, e5m2, q,
                   scales);
}

cudaError_t launch_f8_dequant(const uint8_t* q, const uint8_t* scales, int64_t rows, int cols,
                              int e5m2, bf16* x, cudaStream_t s) {
  const int64_t vecs = rows * (cols >> 4);
  count_launch();
  return ff_launch(k_f8_dequant, grid_for((vecs + 255) / 256), 256, 0, 0, s, q, scales, rows, cols,
                   e5m2, x);
}

}  // namespace alx
