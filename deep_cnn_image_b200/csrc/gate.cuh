// gate.cuh -- the gated block's activations: a(g) and a'(g) in fp32.
//
// Both smooth ones are g times a logistic function p = 1 / (1 + exp(-z)):
// silu with z = g, and gelu's tanh form with z = 2 sqrt(2/pi) (g + 0.044715
// g^3), since (1 + tanh(z/2)) / 2 = p.  So
//   a = g p,   a' = p + g p (1 - p) z'(g).
// exp and the quotient are the fast forms (a few 2^-23 relative, far below
// the 2^-8 of the bf16 results; past z = -87, where 1 + exp(-z) leaves the
// quotient's range, p is 0, and a is off by less than 1e-35).  No infinity meets
// a zero for finite g: z' is evaluated at g cut to 16 in magnitude, past which
// p (1 - p) is 0.  A NaN stays one.
#pragma once
#include <cstdint>

namespace alx {

constexpr float GELU_Z1 = 1.5957691216057308f;               // 2 sqrt(2/pi)
constexpr float GELU_Z3 = 0.044715f * 1.5957691216057308f;

__device__ __forceinline__ float logistic(float z) {
  return __fdividef(1.f, 1.f + __expf(-z));
}

// act: 0 silu, 1 gelu, 2 relu (alexnet_act)
__device__ __forceinline__ float gate_value(float g, int act) {
  if (act == 2) return g <= 0.f ? 0.f : g;
  const float z = act == 0 ? g : g * (GELU_Z1 + GELU_Z3 * g * g);
  return g * logistic(z);
}

__device__ __forceinline__ void gate_both(float g, int act, float& a, float& d) {
  if (act == 2) {
    a = g <= 0.f ? 0.f : g;
    d = g > 0.f ? 1.f : 0.f;
    return;
  }
  float z = g, dz = 1.f;
  if (act == 1) {
    const float c = fminf(fmaxf(g, -16.f), 16.f);
    z = g * (GELU_Z1 + GELU_Z3 * g * g);
    dz = GELU_Z1 + 3.f * GELU_Z3 * c * c;
  }
  const float p = logistic(z);
  a = g * p;
  d = p + a * ((1.f - p) * dz);
}

}  // namespace alx
