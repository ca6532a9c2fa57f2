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

// log(1 + exp(x)) = max(x, 0) + log(1 + e), e = exp(-|x|).  log(1 + e) = e q(e)
// with q a degree-9 Chebyshev interpolant on [0, 1] (relative error below
// 1.5e-7 in fp32 multiply-adds), so small step sizes keep their relative precision without a
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

__device__ __forceinline__ uint32_t shared_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Eight steps of a row on their way into 8 sizeof(T) bytes of shared memory of
// the calling thread's own: asynchronous copies where the row's alignment allows
// them, else through registers (what is at n and behind may come along or not;
// take8 drops it).
template <typename T>
__device__ __forceinline__ void fetch8(T* slot, const T* row, long long t0, int L, int n, bool vec) {
  if (vec && t0 + 8 <= L) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(shared_addr(slot) + 16 * i),
                   "l"((const char*)(row + t0) + 16 * i)
                   : "memory");
    return;
  }
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t0 + i < n)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(shared_addr(slot + i)), "l"(row + t0 + i)
                   : "memory");
      else
        slot[i] = T(0.f);
  } else if (inner8(t0, L)) {
    ldraw8_any(row + t0, *reinterpret_cast<Raw8<T>*>(slot));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) slot[i] = t0 + i < n ? row[t0 + i] : T(0.f);
  }
}
__device__ __forceinline__ void fetched() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// The slot's steps as floats, zeros at n and behind.
template <typename T>
__device__ __forceinline__ void take8(const T* slot, long long t0, int n, float (&v)[8]) {
  Raw8<T> r = *reinterpret_cast<const Raw8<T>*>(slot);
  unpack8(r, v);
  if (t0 + 8 > n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t0 + i >= n) v[i] = 0.f;
  }
}

// The two words below are read again only behind a block barrier, so the
// compiler is told of no memory: the next states' loads may pass the store.
__device__ __forceinline__ void put_shared(uint32_t at, float v) {
  asm volatile("st.shared.f32 [%0], %1;" ::"r"(at), "f"(v));
}
__device__ __forceinline__ void put_global(bool on, float* p, float v) {
  asm volatile("{ .reg .pred q; setp.ne.s32 q, %0, 0; @q st.global.f32 [%1], %2; }" ::"r"((int)on), "l"(p), "f"(v));
}

// Long sequences of few channels are cut into segments of `blocks` 64-step
// blocks, so that the SMs fill.  The states entering the segments come first:
//   scan_ends_kernel sums, for every segment, what its steps leave at its end
//     (backward: at its start) without an entering state, and its step sizes;
//   join_segments_kernel turns those into the entering states.
struct Segments {
  int count, blocks;  // segments of a row; 64-step blocks of a segment
  float* state;       // B x H x count x N (null: one segment)
  float* dt;          // B x H x count
};
cudaError_t launch_segment_states(const ScanArgs& p, const Segments& sg, const float* outer, bool back, int dtype,
                                  cudaStream_t st);
// Time (us) of `blocks` 64-step blocks in `ctas` thread blocks, `most` at once on
// an SM: c + d r for 2048 steps with r of them on an SM, as measured.
inline float scan_cost(long long ctas, int blocks, int most, float c, float d, int sms) {
  const long long r = (ctas + sms - 1) / sms, full = r / most, rest = r % most;
  return (full * (c + most * d) + (rest ? c + rest * d : 0.f)) * blocks / 32;
}
// That of the kernels that find the states entering `count` segments (32 channels
// a thread block) with their launches.  For 1920 thread blocks of 512 steps it gives
// 183 us where 151 were measured, so segments are charged a little more than they cost.
inline float ends_cost(int B, int H, int G, int N, int count, int blocks, int sms) {
  const int chunks = (N + 15) / 16;  // the other times are those of 16 states
  const long long ctas = (long long)B * G * ((H / G + 31) / 32) * (count - 1) * chunks;
  return scan_cost(ctas, blocks, 4, 110.f, 20.f, sms) / chunks + 8.f;
}
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }
inline size_t segments_bytes(const Segments& s, int B, int H, int N) {
  return s.count > 1 ? up256((size_t)B * H * s.count * N * 4) + up256((size_t)B * H * s.count * 4) : 0;
}
inline void place_segments(Segments* s, void* workspace, int B, int H, int N) {
  if (s->count > 1) {
    s->state = (float*)workspace;
    s->dt = (float*)((char*)workspace + up256((size_t)B * H * s->count * N * 4));
  }
}

}  // namespace fc
