// Rows of a sequence tensor for the selective-SSM kernels: eight time steps
// per thread, loaded and stored as 16-byte vectors where a row allows it.
#pragma once

#include <limits.h>

#include "common.cuh"

namespace fc {

constexpr int kVec = 8;  // time steps per thread and load

// Guarded element loads here are plain ones: the headers' __ldg of a 16-bit type
// is an assembly statement without side effects, which the compiler may move out
// of its condition (a null or out-of-range address is then read).

// A B x H x L (or B x G x N x L) tensor with contiguous time: element strides of
// a batch, of a row and of a group; vec = every row starts on a 16-byte boundary.
struct Rows {
  const void* p;
  long long bs, rs, gs;
  int vec;
};

template <typename T> struct Raw8;  // eight elements as loaded
template <> struct Raw8<float> { float4 a, b; };
template <> struct Raw8<__half> { uint4 a; };
template <> struct Raw8<__nv_bfloat16> { uint4 a; };

__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
  v[0] = r.a.x; v[1] = r.a.y; v[2] = r.a.z; v[3] = r.a.w;
  v[4] = r.b.x; v[5] = r.b.y; v[6] = r.b.z; v[7] = r.b.w;
}
__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // a bfloat16 is the upper half of a float
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void ldraw8(const float* p, Raw8<float>& r) {
  r.a = __ldg(reinterpret_cast<const float4*>(p));
  r.b = __ldg(reinterpret_cast<const float4*>(p) + 1);
}
template <typename T>
__device__ __forceinline__ void ldraw8(const T* p, Raw8<T>& r) {
  r.a = __ldg(reinterpret_cast<const uint4*>(p));
}

// Eight 16-bit elements from an address on a two-byte boundary: the two aligned
// vectors around them, moved down by the address's offset in the first.  Both have
// to lie in the row (see inner8).  In two halves, so that several rows' loads can be
// on their way together.
template <typename T>
struct Wide {
  uint4 a, b;
  __device__ __forceinline__ void load(const T* p) {
    const uint4* q = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(p) & ~(uintptr_t)15);
    a = __ldg(q);
    b = __ldg(q + 1);
  }
  __device__ __forceinline__ void put(T* slot, const T* p) const {  // eight elements at a 16-byte boundary
    const uint32_t m = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = m & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = m & 4 ? w[i + 1] : w[i];
    const uint32_t sh = (m & 2) * 8;
    *reinterpret_cast<uint4*>(slot) =
        make_uint4(__funnelshift_r(w[0], w[1], sh), __funnelshift_r(w[1], w[2], sh), __funnelshift_r(w[2], w[3], sh),
                   __funnelshift_r(w[3], w[4], sh));
  }
};
template <typename T>
__device__ __forceinline__ void ldraw8_any(const T* p, Raw8<T>& r) {
  static_assert(sizeof(T) == 2, "two 16-byte vectors hold eight 16-bit elements at any offset");
  Wide<T> w;
  w.load(p);
  w.put(reinterpret_cast<T*>(&r), p);
}
__device__ __forceinline__ bool inner8(long long t0, int L) { return t0 >= 8 && t0 + 16 <= L; }

// Elements t0 .. t0 + 7 of a row of length L as floats; those at n and behind
// it (n <= L) are zero whatever memory holds there.
template <typename T>
__device__ __forceinline__ void load8(const T* row, long long t0, int L, int n, bool vec, float (&v)[8]) {
  if (vec ? t0 + 8 <= L : sizeof(T) == 2 && inner8(t0, L)) {
    Raw8<T> r;
    if constexpr (sizeof(T) == 2) {
      if (vec)
        ldraw8(row + t0, r);
      else
        ldraw8_any(row + t0, r);
    } else {
      ldraw8(row + t0, r);
    }
    unpack8(r, v);
    if (t0 + 8 > n) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t0 + i >= n) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = t0 + i < n ? IO<T>::ldplain(row + t0 + i) : 0.f;
  }
}

__device__ __forceinline__ void stvec8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void stvec8(__half* p, const float (&v)[8]) {
  uint4 o;
  uint32_t* w = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = o;
}
__device__ __forceinline__ void stvec8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 o;
  uint32_t* w = &o.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = o;
}

// Two neighbouring elements, and eight 16-bit ones from an address on a
// two-byte boundary: as 4-byte words, with single elements at both ends where the
// first is not on a 4-byte boundary.
__device__ __forceinline__ void st2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void st2(__half* p, float a, float b) {
  *reinterpret_cast<__half2*>(p) = __floats2half2_rn(a, b);
}
__device__ __forceinline__ void st2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}
template <typename T>
__device__ __forceinline__ void st8_any(T* p, const float (&v)[8]) {
  if (reinterpret_cast<uintptr_t>(p) & 2) {
    IO<T>::st(p, v[0]);
    st2(p + 1, v[1], v[2]);
    st2(p + 3, v[3], v[4]);
    st2(p + 5, v[5], v[6]);
    IO<T>::st(p + 7, v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) st2(p + 2 * i, v[2 * i], v[2 * i + 1]);
  }
}

// Store v at t0 .. t0 + 7 of an output row of length L (zeros at n and behind).
template <typename T>
__device__ __forceinline__ void store8(T* row, long long t0, int L, int n, bool vec, float (&v)[8]) {
  if (t0 + 8 > n) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (t0 + i >= n) v[i] = 0.f;
  }
  if (vec && t0 + 8 <= L) {
    stvec8(row + t0, v);
    return;
  }
  if constexpr (sizeof(T) == 2) {
    if (t0 + 8 <= L) {
      st8_any(row + t0, v);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (t0 + i < L) IO<T>::st(row + t0 + i, v[i]);
}

// lengths[b] clamped to [0, L]; L without lengths.
__device__ __forceinline__ int row_length(const int* lengths, int b, int L) {
  return lengths ? min(max(__ldg(lengths + b), 0), L) : L;
}

// 2^x and 1 / x by the special function unit (relative errors of 2^-22 and 2^-23;
// results below 2^-126 are zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// Two sums or products at once (fp32 pairs of neighbouring registers).
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }

// Sigmoid, SiLU x s(x) and its derivative.  exp(-x) = infinity for x < -88 gives s = 0.
__device__ __forceinline__ float2 sigmoid2(float2 x) {
  const float2 e = mul2(x, both(-kLog2e));
  const float2 d = add2(make_float2(ex2(e.x), ex2(e.y)), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}
__device__ __forceinline__ float2 silu2(float2 x) { return mul2(x, sigmoid2(x)); }
__device__ __forceinline__ float2 dsilu2(float2 x) {
  const float2 s = sigmoid2(x);  // s (1 + x (1 - s))
  return mul2(s, fma2(x, fma2(s, both(-1.f), both(1.f)), both(1.f)));
}
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(x * -kLog2e)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ float dsilu(float x) {
  const float s = sigmoid(x);
  return s * fmaf(x, 1.f - s, 1.f);
}
__device__ __forceinline__ float2 pair(const float (&v)[8], int i) { return make_float2(v[2 * i], v[2 * i + 1]); }

// Row b of a decode batch: its place in the state pool, or -1 for a padded row
// (a slot outside [0, S), or one that an earlier row of the batch holds).
// Every thread of the block calls it.
__device__ __forceinline__ int batch_slot(const int* slots, int b, int S) {
  if (!slots) return b;
  const int slot = __ldg(slots + b);
  bool taken = slot < 0 || slot >= S;
  for (int i = threadIdx.x; i < b; i += blockDim.x) taken |= __ldg(slots + i) == slot;
  return __syncthreads_or(taken) ? -1 : slot;
}

}  // namespace fc
