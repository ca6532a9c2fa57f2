// Selective scan: arguments and the pieces that its kernels share.
#pragma once

#include "rows.cuh"

namespace fc {

// States entering the blocks of this many steps are kept for the backward pass.
constexpr int kCkptSteps = 64;

struct ScanArgs {
  Rows u, delta, z, dy;  // B x H x L (z.p null: no gate)
  Rows Bt, Ct;           // B x (G * N) x L
  const float* A;        // H x N
  const float* D;        // H or null
  const float* dt_bias;  // H or null
  const int* lengths;    // B or null
  const float* state_in; // B x H x N or null
  int B, H, L, N, G;
  int softplus, out_vec;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two products or sums at once (fp32 pairs of neighbouring registers).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }

constexpr float kLog2e = 1.4426950408889634f;

// log(1 + exp(x)) = max(x, 0) + log(1 + e), e = exp(-|x|).  log(1 + e) = e q(e)
// with q a degree-9 Chebyshev interpolant on [0, 1] (relative error below
// 1.2e-7 in fp32), so small step sizes keep their relative precision without a
// branch.
__device__ __forceinline__ float2 softplus2(float2 x) {
  const float2 e = make_float2(ex2(fabsf(x.x) * -kLog2e), ex2(fabsf(x.y) * -kLog2e));
  float2 q = both(-0.003176057f);
  q = fma2(q, e, both(0.019542526f));
  q = fma2(q, e, both(-0.05637361f));
  q = fma2(q, e, both(0.10543624f));
  q = fma2(q, e, both(-0.15269667f));
  q = fma2(q, e, both(0.19663274f));
  q = fma2(q, e, both(-0.24951616f));
  q = fma2(q, e, both(0.3332971f));
  q = fma2(q, e, both(-0.49999893f));
  q = fma2(q, e, both(1.f));
  return fma2(q, e, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return softplus2(both(x)).x; }

}  // namespace fc
