// ff.h -- launchers of the feed-forward operators (norm, 8-bit rows, gated
// block).  All run asynchronously on the stream given and return the launch's
// error; the callers (ff_ops.cu) have checked every argument.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace alx {

using bf16 = __nv_bfloat16;

// the attributes of the device that is current (cached per device)
int ff_num_sms();

// rmsnorm.cu
constexpr int RMSNORM_MAX_COLS = 65536;
cudaError_t launch_rmsnorm_fwd(const bf16* x, const bf16* res, const float* gamma, int64_t rows,
                               int cols, float eps, bf16* sum, bf16* y, float* rstd, uint8_t* q,
                               uint8_t* scales, cudaStream_t s);
// rows of the partial dgamma sums that launch_rmsnorm_bwd writes
int rmsnorm_bwd_parts(int64_t rows, int cols);
cudaError_t launch_rmsnorm_bwd(const bf16* dy, const bf16* dsum, const bf16* sum,
                               const float* gamma, const float* rstd, int64_t rows, int cols,
                               bf16* dx, float* dgamma, float* parts, cudaStream_t s);
cudaError_t launch_f8_quant(const bf16* x, int64_t rows, int cols, int e5m2, uint8_t* q,
                            uint8_t* scales, cudaStream_t s);
cudaError_t launch_f8_dequant(const uint8_t* q, const uint8_t* scales, int64_t rows, int cols,
                              int e5m2, bf16* x, cudaStream_t s);

// gated.cu
// What the backward pass finds of the projections: one of the three.
struct GateSave {
  float* f32;     // [B, 2F]
  bf16* b16;      // [B, 2F]
  uint8_t* q;     // two 8-bit matrices [B, F], one after the other,
  uint8_t* qs;    // and their scales
};
// z fp32 [B, 2F] -> h, and z in what `save` holds
cudaError_t launch_gate_fwd(const float* z, int B, int F, int act, bf16* h, const GateSave& save,
                            cudaStream_t s);
// dz bf16 [B, 2F] from dh and the saved projections
cudaError_t launch_gate_bwd(const bf16* dh, const GateSave& save, int B, int F, int act, bf16* dz,
                            cudaStream_t s);

}  // namespace alx
