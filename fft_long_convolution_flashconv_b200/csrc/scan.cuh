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

// log(1 + exp(x)); x itself above 20, where they agree in fp32.
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(__expf(x)); }

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace fc
