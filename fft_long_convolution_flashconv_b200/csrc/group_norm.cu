// Group norm of each token on its own (so a causal model stays causal) with
// SiLU: what a mixer's output goes through, one group a head.
//
//   xh = (x - mean) rstd over the C / G channels of a group of one token
//   n = xh w + bias,  y = silu(n), or n silu(gate) with a gate
//
// x and gate are B x L x C (a mixer's output) or B x C x L (a scan's output);
// y is B x L x C for the output projection.  The floor is bytes: every kernel
// reads each input once, keeps a group's values in registers for the mean, the
// sum of squares around it and the output, and writes once.  Measured in fp16:
// 16384 tokens of 12 groups of 64 channels 17 us forward and 28 us backward (floors
// 8 and 12; a lane has eight elements to carry a group's sums and reciprocals: 24
// and 39 instructions an element), 65536 tokens of 40 groups of 64 with a gate from
// B x C x L 283 us (floor 154; passes through shared memory).
#include "kernels.cuh"
#include "rows.cuh"

namespace fc {
namespace {

constexpr int kThreads = 256;
// Blocks of the backward pass on an SM: 128 registers a thread (three with 80 spill: 48.6 us against 45.8 for a
// training step on 16384 tokens of 12 groups of 64 in fp16).
constexpr int kBwdBlocks = 2;

struct NormArgs {
  const void *x, *gate, *dy;
  const float *w, *bias;
  long long tokens;  // B * L
  int L, C, G, M;    // M = C / G
  float eps, per;    // per = 1 / M
  int vec;
};

// ------------------------------------------------------------------ B x L x C
// Sum over the P lanes of a group (P <= 32), or over the block (BLOCK).
template <bool BLOCK>
__device__ __forceinline__ float sum_unit(float v, int P, float* red) {
  if (BLOCK) {
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += red[i];
  } else {
    for (int d = P >> 1; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
  }
  return v;
}

// Eight channels m .. m + 7 of a group of M (zeros behind it).
template <typename T>
__device__ __forceinline__ void ld_group(const T* base, int m, int M, bool vec, float (&v)[8]) {
  load8(base, m, M, m < M ? M : 0, vec, v);
}
template <typename T>
__device__ __forceinline__ void st_group(T* base, int m, int M, bool vec, float (&v)[8]) {
  if (m < M) store8(base, m, M, M, vec, v);
}
__device__ __forceinline__ void ld_param(const float* p, int m, int M, float other, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p && m + i < M ? __ldg(p + m + i) : other;
}

// Mean and rstd of a group; FULL: every lane's vectors lie inside it.
template <bool BLOCK, bool FULL, int V>
__device__ __forceinline__ void stats(float2 (&x)[V][4], int lane, int P, const NormArgs& p, float* red, float& mean,
                                      float& rstd) {
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) s = add2(s, x[v][i]);
  mean = sum_unit<BLOCK>(s.x + s.y, P, red) * p.per;
  s = make_float2(0.f, 0.f);
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 d = add2(x[v][i], both(-mean));
      if (!FULL) {
        const int m = (v * P + lane) * 8 + 2 * i;
        d = make_float2(m < p.M ? d.x : 0.f, m + 1 < p.M ? d.y : 0.f);
      }
      s = fma2(d, d, s);
      x[v][i] = d;  // x - mean from here on, zero behind the group
    }
  rstd = rsqrtf(fmaf(sum_unit<BLOCK>(s.x + s.y, P, red), p.per, p.eps));
}

// P lanes (or the block) share a group of one token, V vectors of eight channels
// each.  The groups of all tokens, in memory order, are dealt out to the blocks
// kThreads / P at a time; the number of blocks makes the stride a multiple of G, so
// that a thread keeps its channels, and their weights in registers.  The next
// group's values are loaded while the present one is worked on.
template <typename T, int V>
struct Group {
  Raw8<T> r[V];
  __device__ __forceinline__ void get(int v, float2 (&x)[4]) const {
    float a[8];
    unpack8(r[v], a);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = pair(a, i);
  }
  template <bool FULL>
  __device__ __forceinline__ void load(const void* base, long long off, int lane, int P, int M, bool vec, bool on) {
    const T* q = (const T*)base + off;
    if (FULL && vec) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        r[v] = Raw8<T>{};
        if (on) ldraw8(q + (v * P + lane) * 8, r[v]);
      }
      return;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int m = (v * P + lane) * 8;
      T* e = reinterpret_cast<T*>(&r[v]);
      if (on && vec && m + 8 <= M) {
        ldraw8(q + m, r[v]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = on && m + i < M ? q[m + i] : T(0.f);
      }
    }
  }
};

template <typename T, int V, bool BLOCK, bool FULL, bool GATE>
__global__ __launch_bounds__(kThreads, V == 1 ? 4 : 1) void norm_kernel(NormArgs p, T* y, int P) {
  __shared__ float red[kThreads / 32];
  const int lane = threadIdx.x % P, M = p.M;
  const long long units = p.tokens * p.G, subs = kThreads / P, stride = gridDim.x * subs;
  const long long first = blockIdx.x * subs;
  long long unit = first + threadIdx.x / P;
  const long long g = unit % p.G;
  float2 w[V][4], bias[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8];
    ld_param(p.w ? p.w + g * M : nullptr, (v * P + lane) * 8, M, 1.f, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[v][i] = pair(a, i);
    ld_param(p.bias ? p.bias + g * M : nullptr, (v * P + lane) * 8, M, 0.f, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[v][i] = pair(a, i);
  }
  long long off = unit * M;
  const long long step = stride * M;
  Group<T, V> xn, zn;
  xn.template load<FULL>(p.x, off, lane, P, M, p.vec, unit < units);
  if (GATE) zn.template load<FULL>(p.gate, off, lane, P, M, p.vec, unit < units);
  for (long long base = first; base < units; base += stride, unit += stride, off += step) {  // alike for the block
    float2 x[V][4], z[V][4];
    float mean, rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      xn.get(v, x[v]);
      if (GATE) zn.get(v, z[v]);
    }
    const bool more = unit + stride < units;
    xn.template load<FULL>(p.x, off + step, lane, P, M, p.vec, more);
    if (GATE) zn.template load<FULL>(p.gate, off + step, lane, P, M, p.vec, more);
    stats<BLOCK, FULL, V>(x, lane, P, p, red, mean, rstd);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 n = fma2(mul2(x[v][i], both(rstd)), w[v][i], bias[v][i]);
        const float2 a = GATE ? mul2(n, silu2(z[v][i])) : silu2(n);
        o[2 * i] = a.x;
        o[2 * i + 1] = a.y;
      }
      if (unit < units) st_group(y + off, (v * P + lane) * 8, M, p.vec, o);
    }
  }
}

// Backward.  dn = dy silu'(n) (dy silu(gate) with a gate), e = dn w,
//   dx = rstd (e - mean(e) - xh mean(e xh)),  dw = sum dn xh,  dbias = sum dn.
// Dealt out as above; a thread sums its channels' dw and dbias in registers, the
// block adds its threads of one group in order, norm_sum_kernel the blocks.
template <typename T, int V, bool BLOCK, bool FULL, bool GATE>
__global__ __launch_bounds__(kThreads, V == 1 ? kBwdBlocks : 1) void norm_bwd_kernel(NormArgs p, T* dx, T* dgate, float* part,
                                                                            int P) {
  __shared__ float red[kThreads / 32];
  __shared__ float acc[kThreads * 8 * V];
  const int lane = threadIdx.x % P, sub = threadIdx.x / P, M = p.M;
  const int subs = kThreads / P;
  const long long units = p.tokens * p.G, stride = (long long)gridDim.x * subs;
  const long long first = (long long)blockIdx.x * subs;
  long long unit = first + sub;
  const long long g = unit % p.G;
  float2 w[V][4], bias[V][4], dw[V][4], db[V][4];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a[8];
    ld_param(p.w ? p.w + g * M : nullptr, (v * P + lane) * 8, M, 1.f, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[v][i] = pair(a, i);
    ld_param(p.bias ? p.bias + g * M : nullptr, (v * P + lane) * 8, M, 0.f, a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bias[v][i] = pair(a, i);
      dw[v][i] = db[v][i] = make_float2(0.f, 0.f);
    }
  }
  Group<T, V> xn, yn, zn;
  long long off = unit * M;
  const long long step = stride * M;
  auto load = [&](long long at, bool on) {
    xn.template load<FULL>(p.x, at, lane, P, M, p.vec, on);
    yn.template load<FULL>(p.dy, at, lane, P, M, p.vec, on);
    if (GATE) zn.template load<FULL>(p.gate, at, lane, P, M, p.vec, on);
  };
  load(off, unit < units);
  for (long long base = first; base < units; base += stride, unit += stride, off += step) {
    const bool live = unit < units;
    float2 x[V][4], dn[V][4], z[V][4];
    float mean, rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      xn.get(v, x[v]);
      yn.get(v, dn[v]);
      if (GATE) zn.get(v, z[v]);
    }
    load(off + step, unit + stride < units);
    stats<BLOCK, FULL, V>(x, lane, P, p, red, mean, rstd);
    float2 se = make_float2(0.f, 0.f), sex = se;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 xh = mul2(x[v][i], both(rstd)), n = fma2(xh, w[v][i], bias[v][i]);
        x[v][i] = xh;
        if (GATE) {
          const float2 s = sigmoid2(z[v][i]), zs = mul2(z[v][i], s);
          // dy n s (1 + z (1 - s))
          const float2 slope = mul2(s, fma2(z[v][i], fma2(s, both(-1.f), both(1.f)), both(1.f)));
          const float2 d = mul2(mul2(dn[v][i], n), slope);
          o[2 * i] = d.x;
          o[2 * i + 1] = d.y;
          dn[v][i] = mul2(dn[v][i], zs);
        } else {
          dn[v][i] = mul2(dn[v][i], dsilu2(n));
        }
        dw[v][i] = fma2(dn[v][i], xh, dw[v][i]);
        db[v][i] = add2(db[v][i], dn[v][i]);
        dn[v][i] = mul2(dn[v][i], w[v][i]);  // e from here on
        se = add2(se, dn[v][i]);
        sex = fma2(dn[v][i], xh, sex);
      }
      if (GATE && live) st_group(dgate + off, (v * P + lane) * 8, M, p.vec, o);
    }
    const float me = sum_unit<BLOCK>(se.x + se.y, P, red) * p.per, mex = sum_unit<BLOCK>(sex.x + sex.y, P, red) * p.per;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = mul2(both(rstd), fma2(x[v][i], both(-mex), add2(dn[v][i], both(-me))));
        o[2 * i] = d.x;
        o[2 * i + 1] = d.y;
      }
      if (live) st_group(dx + off, (v * P + lane) * 8, M, p.vec, o);
    }
  }
  const int groups = subs < p.G ? subs : p.G;  // this block's groups: those of its first units
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 a = which ? db[v][i / 2] : dw[v][i / 2];
        acc[sub * (P * 8 * V) + (v * P + lane) * 8 + i] = i & 1 ? a.y : a.x;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < groups * M; i += kThreads) {
      float s = 0.f;
      for (int k = i / M; k < subs; k += p.G) s += acc[k * (P * 8 * V) + i % M];
      part[((long long)blockIdx.x * 2 + which) * groups * M + i] = s;
    }
  }
}

// dw and dbias from the blocks' parts, in order.  Block j's part holds `groups`
// groups from (j first) % G on; a channel's sum is split over 32 threads.
__global__ void norm_sum_kernel(const float* part, float* dw, float* dbias, int C, int M, int G, int groups, int first,
                                int blocks) {
  __shared__ float red[8][33];
  const int cc = threadIdx.x % 8, row = threadIdx.x / 8;  // 8 channels, 32 rows of blocks
  const int i = blockIdx.x * 8 + cc;
  float v = 0.f;
  if (i < 2 * C) {
    const int which = i / C, g = i % C / M, m = i % C % M, back = (int)(32LL * first % G);
    int k = (int)(((long long)g + G - (long long)row * first % G) % G);  // the group's place in part `row`
#pragma unroll 4
    for (int j = row; j < blocks; j += 32) {
      if (k < groups) v += part[((long long)j * 2 + which) * groups * M + (long long)k * M + m];
      k -= back;
      if (k < 0) k += G;
    }
  }
  red[cc][row] = v;
  __syncthreads();
  if (row == 0 && i < 2 * C) {
    v = 0.f;
    for (int j = 0; j < 32; ++j) v += red[cc][j];
    if (i < C) {
      if (dw) dw[i] = v;
    } else if (dbias) {
      dbias[i - C] = v;
    }
  }
}

// ------------------------------------------------------------------ B x C x L
// A block takes 64 tokens of a group.  A thread holds eight tokens (one 16-byte
// access of a channel's row) of V channels at a time: two neighbouring ones of
// every 64 (V = 1: every 32nd).  Sums over the channels go over shuffles and shared
// memory.  Token-major rows (y, dy) pass through a shared tile of 64 tokens by
// 32 V channels whose vectors of eight channels are swizzled by the token, so that
// both directions of the transposition touch all banks: a warp's eight token
// vectors by four channel pairs are 32 words of eight different vectors.
constexpr int TT = 64;

template <int V>
__device__ __forceinline__ int channel_of(int j) {  // j-th of a thread's channels in a slab
  const int mq = threadIdx.x >> 3;
  return V == 1 ? mq : j / 2 * 64 + mq * 2 + j % 2;
}
template <int V>
__device__ __forceinline__ int tile_pos(int t, int m) {  // row of at least 64 channels: eight vectors
  constexpr int W = 32 * V < 64 ? 64 : 32 * V;
  return t * W + ((((m >> 3) & ~7) | (((m >> 3) ^ (t >> 3)) & 7)) << 3) + (m & 7);
}
template <int V> constexpr size_t tile_elems() { return (size_t)TT * (32 * V < 64 ? 64 : 32 * V); }

__device__ __forceinline__ float2 ld2(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ float2 ld2(const __half* p) { return __half22float2(*reinterpret_cast<const __half2*>(p)); }
__device__ __forceinline__ float2 ld2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}

// Sums over all 32 channel threads of the eight tokens that a thread holds, by way
// of red[32][kRed]: four neighbouring threads add up a token, rows four apart each
// (kRed = 8 mod 32 words keeps them on different banks).
constexpr int kRed = TT + 8;

__device__ __forceinline__ void sum_tokens(float (&s)[8], float (*red)[kRed]) {
  const int tv = threadIdx.x & 7, mq = threadIdx.x >> 3, t = threadIdx.x >> 2, q = threadIdx.x & 3;
  __syncthreads();
  *reinterpret_cast<float4*>(&red[mq][tv * 8]) = make_float4(s[0], s[1], s[2], s[3]);
  *reinterpret_cast<float4*>(&red[mq][tv * 8 + 4]) = make_float4(s[4], s[5], s[6], s[7]);
  __syncthreads();
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) v += red[q + 4 * i][t];
  v += __shfl_xor_sync(~0u, v, 1);
  v += __shfl_xor_sync(~0u, v, 2);
  __syncwarp();
  if (q == 0) red[0][t] = v;  // this warp alone reads the column
  __syncthreads();
  const float4 a = *reinterpret_cast<const float4*>(&red[0][tv * 8]);
  const float4 b = *reinterpret_cast<const float4*>(&red[0][tv * 8 + 4]);
  s[0] = a.x; s[1] = a.y; s[2] = a.z; s[3] = a.w;
  s[4] = b.x; s[5] = b.y; s[6] = b.z; s[7] = b.w;
}

template <typename T, int V>
struct Slab {  // the rows of a group that a block works on
  const NormArgs& p;
  long long row0;  // of the group's first channel
  int t0;          // first token of the thread
  __device__ __forceinline__ void load(const void* a, int m0, float (&v)[V][8]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int m = m0 + channel_of<V>(j);
      load8((const T*)a + (row0 + (m < p.M ? m : 0)) * p.L, t0, p.L, m < p.M ? p.L : 0, p.vec, v[j]);
    }
  }
  __device__ __forceinline__ void store(void* a, int m, float (&v)[8]) const {
    if (m < p.M && t0 < p.L) store8((T*)a + (row0 + m) * p.L, t0, p.L, p.L, p.vec, v);
  }
};

// Mean and rstd of the thread's eight tokens; x holds the slab on return where there is only one.
template <typename T, int V>
__device__ __forceinline__ void stats_cm(const Slab<T, V>& sl, int M, float eps, float (&x)[V][8], float (*red)[kRed],
                                         float (&mean)[8], float (&rstd)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) mean[i] = rstd[i] = 0.f;
  for (int m0 = 0; m0 < M; m0 += 32 * V) {
    sl.load(sl.p.x, m0, x);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) mean[i] += x[j][i];
  }
  sum_tokens(mean, red);
#pragma unroll
  for (int i = 0; i < 8; ++i) mean[i] *= sl.p.per;
  for (int m0 = 0; m0 < M; m0 += 32 * V) {
    if (M > 32 * V) sl.load(sl.p.x, m0, x);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (m0 + channel_of<V>(j) < M)
#pragma unroll
        for (int i = 0; i < 8; ++i) rstd[i] = fmaf(x[j][i] - mean[i], x[j][i] - mean[i], rstd[i]);
  }
  sum_tokens(rstd, red);
#pragma unroll
  for (int i = 0; i < 8; ++i) rstd[i] = rsqrtf(fmaf(rstd[i], sl.p.per, eps));
}

// Vectors of eight channels of a slab's token-major rows, dealt out to the block:
// f(token of the tile, first channel of the slab) for each.
template <int V, typename F>
__device__ __forceinline__ void each_vector(int width, F f) {
  if (width == 32 * V) {
#pragma unroll
    for (int k = 0; k < TT * 4 * V / kThreads; ++k) {
      const int i = threadIdx.x + k * kThreads;
      f(i / (4 * V), i % (4 * V) * 8);
    }
  } else {
    const int chunks = (width + 7) / 8;
    for (int i = threadIdx.x; i < TT * chunks; i += kThreads) f(i / chunks, i % chunks * 8);
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads, V <= 2 ? 2 : 1) void norm_cm_kernel(NormArgs p, T* y, int tiles) {
  extern __shared__ float4 smem4[];
  T* tile = reinterpret_cast<T*>(smem4);
  __shared__ __align__(16) float red[32][kRed];
  const int bg = blockIdx.x / tiles, tl = blockIdx.x - bg * tiles, b = bg / p.G, g = bg - b * p.G;
  const int M = p.M, tv = threadIdx.x & 7, tb = tl * TT;
  const Slab<T, V> sl{p, (long long)b * p.C + g * M, tb + tv * 8};
  float x[V][8], z[V][8], mean[8], rstd[8];
  const bool one = M <= 32 * V;
  if (one && p.gate) sl.load(p.gate, 0, z);
  stats_cm<T, V>(sl, M, p.eps, x, red, mean, rstd);
  for (int m0 = 0; m0 < M; m0 += 32 * V) {
    if (!one) {
      sl.load(p.x, m0, x);
      if (p.gate) sl.load(p.gate, m0, z);
    }
    __syncthreads();  // the tile may still be read
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int m = m0 + channel_of<V>(j);
      const float w = p.w && m < M ? __ldg(p.w + (long long)g * M + m) : 1.f;
      const float bias = p.bias && m < M ? __ldg(p.bias + (long long)g * M + m) : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 d = make_float2(x[j][2 * i] - mean[2 * i], x[j][2 * i + 1] - mean[2 * i + 1]);
        const float2 n = fma2(mul2(d, pair(rstd, i)), both(w), both(bias));
        const float2 a = p.gate ? mul2(n, silu2(pair(z[j], i))) : silu2(n);
        x[j][2 * i] = a.x;
        x[j][2 * i + 1] = a.y;
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (V == 1) {
        IO<T>::st(tile + tile_pos<V>(tv * 8 + i, channel_of<V>(0)), x[0][i]);
      } else {
#pragma unroll
        for (int j = 0; j < V; j += 2) st2(tile + tile_pos<V>(tv * 8 + i, channel_of<V>(j)), x[j][i], x[j + 1][i]);
      }
    }
    __syncthreads();
    const int width = min(32 * V, M - m0);
    each_vector<V>(width, [&](int t, int mm) {
      if (tb + t >= p.L) return;
      T* o = y + ((long long)b * p.L + tb + t) * p.C + (long long)g * M + m0 + mm;
      const T* s = tile + tile_pos<V>(t, mm);
      if (mm + 8 <= width && ((uintptr_t)o & 15) == 0) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(o)[i] = reinterpret_cast<const uint4*>(s)[i];
      } else {
        for (int i = 0; i < 8 && mm + i < width; ++i) o[i] = s[i];
      }
    });
  }
}

// The same for whole tiles: groups of 32 V channels, rows of whole tiles on 16-byte
// boundaries.  Nothing is guarded, the gate stays as loaded until it is used.
template <typename T, int V, bool GATE>
__global__ __launch_bounds__(kThreads, V <= 2 ? 4 : V <= 4 ? 2 : 1) void norm_cm_whole_kernel(NormArgs p, T* y,
                                                                                              int tiles) {
  extern __shared__ float4 smem4[];
  T* tile = reinterpret_cast<T*>(smem4);
  __shared__ __align__(16) float red[32][kRed];
  const int bg = blockIdx.x / tiles, tl = blockIdx.x - bg * tiles, b = bg / p.G, g = bg - b * p.G;
  const int tv = threadIdx.x & 7;
  const long long off = ((long long)b * p.C + (long long)g * p.M) * p.L + tl * TT + tv * 8;
  const T* xp = (const T*)p.x + off + (long long)channel_of<V>(0) * p.L;
  const T* zp = (const T*)p.gate + off + (long long)channel_of<V>(0) * p.L;
  Raw8<T> xr[V], zr[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const long long d = (long long)(V == 1 ? 0 : j / 2 * 64 + j % 2) * p.L;  // channels from the thread's first
    ldraw8(xp + d, xr[j]);
    if (GATE) ldraw8(zp + d, zr[j]);
  }
  float2 mean[4], rstd[4];
  float s[8];
  float2 x[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float v[8];
    unpack8(xr[j], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[j][i] = pair(v, i);
      mean[i] = j == 0 ? x[j][i] : add2(mean[i], x[j][i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[2 * i] = mean[i].x, s[2 * i + 1] = mean[i].y;
  sum_tokens(s, red);
#pragma unroll
  for (int i = 0; i < 4; ++i) mean[i] = mul2(pair(s, i), both(-p.per));
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[j][i] = add2(x[j][i], mean[i]);  // less the mean from here on
      rstd[i] = j == 0 ? mul2(x[j][i], x[j][i]) : fma2(x[j][i], x[j][i], rstd[i]);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[2 * i] = rstd[i].x, s[2 * i + 1] = rstd[i].y;
  sum_tokens(s, red);
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = rsqrtf(fmaf(s[i], p.per, p.eps));
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int m = g * p.M + channel_of<V>(j);
    const float w = p.w ? __ldg(p.w + m) : 1.f, bias = p.bias ? __ldg(p.bias + m) : 0.f;
    float z[8];
    if (GATE) unpack8(zr[j], z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 n = fma2(mul2(x[j][i], pair(s, i)), both(w), both(bias));
      x[j][i] = GATE ? mul2(n, silu2(pair(z, i))) : silu2(n);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (V == 1) {
      IO<T>::st(tile + tile_pos<V>(tv * 8 + i, channel_of<V>(0)), i & 1 ? x[0][i / 2].y : x[0][i / 2].x);
    } else {
#pragma unroll
      for (int j = 0; j < V; j += 2)
        st2(tile + tile_pos<V>(tv * 8 + i, channel_of<V>(j)), i & 1 ? x[j][i / 2].y : x[j][i / 2].x,
            i & 1 ? x[j + 1][i / 2].y : x[j + 1][i / 2].x);
    }
  }
  __syncthreads();
  T* yt = y + ((long long)b * p.L + tl * TT) * p.C + g * p.M;
  each_vector<V>(32 * V, [&](int t, int mm) {
    T* o = yt + (long long)t * p.C + mm;
    const T* q = tile + tile_pos<V>(t, mm);
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(o)[i] = reinterpret_cast<const uint4*>(q)[i];
  });
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void norm_cm_bwd_kernel(NormArgs p, T* dx, T* dgate, float* part, int tiles,
                                                               int per_split) {
  extern __shared__ float4 smem4[];
  float* acc = reinterpret_cast<float*>(smem4);  // [2][M] dw, dbias of the block
  const int Ma = (p.M + 3) / 4 * 4;
  T* tile = reinterpret_cast<T*>(acc + 2 * Ma);
  __shared__ __align__(16) float red[32][kRed];
  const int g = blockIdx.x, M = p.M, tv = threadIdx.x & 7;
  const long long items = p.tokens / p.L * tiles;  // (batch row, tile of tokens)
  const long long lo = (long long)blockIdx.y * per_split, hi = lo + per_split < items ? lo + per_split : items;
  for (int i = threadIdx.x; i < 2 * Ma; i += kThreads) acc[i] = 0.f;
  for (long long it = lo; it < hi; ++it) {
    const long long b = it / tiles;
    const int tb = (int)(it % tiles) * TT;
    const Slab<T, V> sl{p, b * p.C + (long long)g * M, tb + tv * 8};
    float x[V][8], mean[8], rstd[8], se[8], sex[8];
    stats_cm<T, V>(sl, M, p.eps, x, red, mean, rstd);
#pragma unroll
    for (int i = 0; i < 8; ++i) se[i] = sex[i] = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      for (int m0 = 0; m0 < M; m0 += 32 * V) {
        const int width = min(32 * V, M - m0);
        if (M > 32 * V || pass == 0) {  // dy of the slab into the tile
          __syncthreads();
          each_vector<V>(width, [&](int t, int mm) {
            T* s = tile + tile_pos<V>(t, mm);
            const T* o = (const T*)p.dy + (b * p.L + tb + t) * p.C + (long long)g * M + m0 + mm;
            if (tb + t < p.L && mm + 8 <= width && ((uintptr_t)o & 15) == 0) {
#pragma unroll
              for (int i = 0; i < (int)sizeof(T) / 2; ++i)
                reinterpret_cast<uint4*>(s)[i] = __ldg(reinterpret_cast<const uint4*>(o) + i);
            } else {
              for (int i = 0; i < 8; ++i)
                if (tb + t < p.L && mm + i < width)
                  s[i] = o[i];
                else
                  IO<T>::st(s + i, 0.f);
            }
          });
          __syncthreads();
        }
        if (M > 32 * V) sl.load(p.x, m0, x);
        float dyv[V][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if constexpr (V == 1) {
            dyv[0][i] = IO<T>::ldplain(tile + tile_pos<V>(tv * 8 + i, channel_of<V>(0)));
          } else {
#pragma unroll
            for (int j = 0; j < V; j += 2) {
              const float2 d = ld2(tile + tile_pos<V>(tv * 8 + i, channel_of<V>(j)));
              dyv[j][i] = d.x;
              dyv[j + 1][i] = d.y;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int m = m0 + channel_of<V>(j);
          const bool ok = m < M;
          const float w = ok && p.w ? __ldg(p.w + (long long)g * M + m) : 1.f;
          const float bias = ok && p.bias ? __ldg(p.bias + (long long)g * M + m) : 0.f;
          float z[8], o[8], dg[8], sw = 0.f, sb = 0.f;
          if (p.gate) load8((const T*)p.gate + (sl.row0 + (ok ? m : 0)) * p.L, sl.t0, p.L, ok ? p.L : 0, p.vec, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = (x[j][i] - mean[i]) * rstd[i];
            const float dy = ok ? dyv[j][i] : 0.f;
            const float n = fmaf(xh, w, bias);
            const float dn = dy * (p.gate ? silu(z[i]) : dsilu(n)), e = dn * w;
            if (pass == 0) {
              se[i] += e;
              sex[i] = fmaf(e, xh, sex[i]);
            } else {
              o[i] = rstd[i] * (e - se[i] - xh * sex[i]);
              if (p.gate) dg[i] = dy * n * dsilu(z[i]);
              sw = fmaf(dn, xh, sw);
              sb += dn;
            }
          }
          if (pass == 1) {
            sl.store(dx, m, o);
            if (p.gate) sl.store(dgate, m, dg);
#pragma unroll
            for (int d = 1; d < 8; d *= 2) {
              sw += __shfl_xor_sync(~0u, sw, d);
              sb += __shfl_xor_sync(~0u, sb, d);
            }
            if (ok && tv == 0) {  // a channel has one such thread
              acc[m] += sw;
              acc[Ma + m] += sb;
            }
          }
        }
      }
      if (pass == 0) {
        sum_tokens(se, red);
        sum_tokens(sex, red);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          se[i] *= p.per;
          sex[i] *= p.per;
        }
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * M; i += kThreads) {
    const int which = i / M, m = i % M;
    part[((long long)blockIdx.y * 2 + which) * p.C + (long long)g * M + m] = acc[which * Ma + m];
  }
}

// ------------------------------------------------------------------ launches
struct Plan {
  int P, V;
  bool block;
};
Plan plan(int M) {
  const int chunks = (M + 7) / 8;
  Plan r{1, 1, false};
  if (chunks <= 128) {
    while (r.P < 32 && r.P < chunks) r.P *= 2;
    while (r.P * r.V < chunks) r.V *= 2;
  } else {
    r.block = true;
    r.P = kThreads;
    while (r.P * r.V < chunks) r.V *= 2;
  }
  return r;
}
int plan_cm(int M) { return M <= 32 ? 1 : M <= 64 ? 2 : M <= 128 ? 4 : 8; }

// Blocks for `units` groups, kThreads / P at a time and each at least `least` times:
// a multiple of G / gcd(G, kThreads / P), so that a thread's group stays the same,
// and no more than `most` or that.
int blocks_of(long long units, int G, int P, int least, int most) {
  const int subs = kThreads / P;
  int a = G, c = subs;
  while (c) {
    const int r = a % c;
    a = c;
    c = r;
  }
  const int whole = G / a;
  long long want = (units + (long long)subs * least - 1) / ((long long)subs * least);
  if (want > most) want = most;
  long long n = want / whole * whole;
  return (int)(n < whole ? whole : n);
}

template <typename T, int V, bool BLOCK>
cudaError_t fwd_v(const NormArgs& p, void* y, int P, cudaStream_t st) {
  const int blocks = blocks_of(p.tokens * p.G, p.G, P, 1, num_sms() * (V == 1 ? 4 : 2));
  constexpr bool FULL = V == 1 && !BLOCK;  // possible: a power of two of 8 to 256 channels
  if (FULL && p.M == P * 8)
    if (p.gate)
      norm_kernel<T, V, BLOCK, FULL, true><<<blocks, kThreads, 0, st>>>(p, (T*)y, P);
    else
      norm_kernel<T, V, BLOCK, FULL, false><<<blocks, kThreads, 0, st>>>(p, (T*)y, P);
  else if (p.gate)
    norm_kernel<T, V, BLOCK, false, true><<<blocks, kThreads, 0, st>>>(p, (T*)y, P);
  else
    norm_kernel<T, V, BLOCK, false, false><<<blocks, kThreads, 0, st>>>(p, (T*)y, P);
  return cudaGetLastError();
}
template <typename T, int V, bool BLOCK>
cudaError_t bwd_v(const NormArgs& p, void* dx, void* dgate, float* part, int P, int blocks, cudaStream_t st) {
  constexpr bool FULL = V == 1 && !BLOCK;
  if (FULL && p.M == P * 8)
    if (p.gate)
      norm_bwd_kernel<T, V, BLOCK, FULL, true><<<blocks, kThreads, 0, st>>>(p, (T*)dx, (T*)dgate, part, P);
    else
      norm_bwd_kernel<T, V, BLOCK, FULL, false><<<blocks, kThreads, 0, st>>>(p, (T*)dx, (T*)dgate, part, P);
  else if (p.gate)
    norm_bwd_kernel<T, V, BLOCK, false, true><<<blocks, kThreads, 0, st>>>(p, (T*)dx, (T*)dgate, part, P);
  else
    norm_bwd_kernel<T, V, BLOCK, false, false><<<blocks, kThreads, 0, st>>>(p, (T*)dx, (T*)dgate, part, P);
  return cudaGetLastError();
}
template <typename T, int V>
cudaError_t fwd_cm(const NormArgs& p, void* y, cudaStream_t st) {
  const int tiles = (p.L + TT - 1) / TT;
  const size_t smem = tile_elems<V>() * sizeof(T);
  // whole tiles, and rows of y on 16-byte boundaries
  if (p.M == 32 * V && p.vec && p.L % TT == 0 && p.C % 8 == 0) {
    const cudaError_t e = p.gate ? smem_optin<norm_cm_whole_kernel<T, V, true>>(smem)
                                 : smem_optin<norm_cm_whole_kernel<T, V, false>>(smem);
    if (e != cudaSuccess) return e;
    const unsigned grid = (unsigned)(p.tokens / p.L * tiles * p.G);
    if (p.gate)
      norm_cm_whole_kernel<T, V, true><<<grid, kThreads, smem, st>>>(p, (T*)y, tiles);
    else
      norm_cm_whole_kernel<T, V, false><<<grid, kThreads, smem, st>>>(p, (T*)y, tiles);
    return cudaGetLastError();
  }
  const cudaError_t e = smem_optin<norm_cm_kernel<T, V>>(smem);
  if (e != cudaSuccess) return e;
  norm_cm_kernel<T, V><<<(unsigned)(p.tokens / p.L * tiles * p.G), kThreads, smem, st>>>(p, (T*)y, tiles);
  return cudaGetLastError();
}
template <typename T, int V>
cudaError_t bwd_cm(const NormArgs& p, void* dx, void* dgate, float* part, int splits, cudaStream_t st) {
  const int tiles = (p.L + TT - 1) / TT;
  const long long items = p.tokens / p.L * tiles;
  const size_t smem = (size_t)(p.M + 3) / 4 * 4 * 8 + tile_elems<V>() * sizeof(T);
  const cudaError_t e = smem_optin<norm_cm_bwd_kernel<T, V>>(smem);
  if (e != cudaSuccess) return e;
  norm_cm_bwd_kernel<T, V><<<dim3(p.G, splits), kThreads, smem, st>>>(p, (T*)dx, (T*)dgate, part, tiles,
                                                                     (int)((items + splits - 1) / splits));
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const NormArgs& p, void* y, int cm, cudaStream_t st) {
  if (cm) switch (plan_cm(p.M)) {
      case 1: return fwd_cm<T, 1>(p, y, st);
      case 2: return fwd_cm<T, 2>(p, y, st);
      case 4: return fwd_cm<T, 4>(p, y, st);
      default: return fwd_cm<T, 8>(p, y, st);
    }
  const Plan r = plan(p.M);
  if (r.block) switch (r.V) {
      case 1: return fwd_v<T, 1, true>(p, y, r.P, st);
      case 2: return fwd_v<T, 2, true>(p, y, r.P, st);
      default: return fwd_v<T, 4, true>(p, y, r.P, st);
    }
  switch (r.V) {
    case 1: return fwd_v<T, 1, false>(p, y, r.P, st);
    case 2: return fwd_v<T, 2, false>(p, y, r.P, st);
    default: return fwd_v<T, 4, false>(p, y, r.P, st);
  }
}
template <typename T>
cudaError_t bwd(const NormArgs& p, void* dx, void* dgate, float* part, int splits, int cm, cudaStream_t st) {
  if (cm) switch (plan_cm(p.M)) {
      case 1: return bwd_cm<T, 1>(p, dx, dgate, part, splits, st);
      case 2: return bwd_cm<T, 2>(p, dx, dgate, part, splits, st);
      case 4: return bwd_cm<T, 4>(p, dx, dgate, part, splits, st);
      default: return bwd_cm<T, 8>(p, dx, dgate, part, splits, st);
    }
  const Plan r = plan(p.M);
  if (r.block) switch (r.V) {
      case 1: return bwd_v<T, 1, true>(p, dx, dgate, part, r.P, splits, st);
      case 2: return bwd_v<T, 2, true>(p, dx, dgate, part, r.P, splits, st);
      default: return bwd_v<T, 4, true>(p, dx, dgate, part, r.P, splits, st);
    }
  switch (r.V) {
    case 1: return bwd_v<T, 1, false>(p, dx, dgate, part, r.P, splits, st);
    case 2: return bwd_v<T, 2, false>(p, dx, dgate, part, r.P, splits, st);
    default: return bwd_v<T, 4, false>(p, dx, dgate, part, r.P, splits, st);
  }
}

}  // namespace

cudaError_t launch_group_norm(const void* x, const float* w, const float* bias, const void* gate, void* y, int B, int L,
                              int C, int G, float eps, int channel_major, int vec, int dtype, cudaStream_t st) {
  const NormArgs p{x, gate, nullptr, w, bias, (long long)B * L, L, C, G, C / G, eps, (float)(1.0 / (C / G)), vec};
  switch (dtype) {
    case 0: return fwd<float>(p, y, channel_major, st);
    case 1: return fwd<__half>(p, y, channel_major, st);
    case 2: return fwd<__nv_bfloat16>(p, y, channel_major, st);
    default: return cudaErrorInvalidValue;
  }
}

namespace {
// Parts of dw and dbias, and the groups of a part.
struct Parts {
  int count, groups, first;
};
Parts parts(int B, int L, int C, int G, int channel_major) {
  if (channel_major) {  // about eight blocks an SM, a whole row of channels a part
    const long long items = (long long)B * ((L + TT - 1) / TT);
    long long s = num_sms() * 8 / G;
    if (s > items) s = items;
    return {(int)(s < 1 ? 1 : s), G, 0};
  }
  const int P = plan(C / G).P, subs = kThreads / P;
  return {blocks_of((long long)B * L * G, G, P, 2, num_sms() * kBwdBlocks), subs < G ? subs : G, subs};
}
}  // namespace

size_t group_norm_bwd_workspace_bytes(int B, int L, int C, int G, int channel_major) {
  const Parts q = parts(B, L, C, G, channel_major);
  return (size_t)q.count * 2 * q.groups * (C / G) * 4;
}

cudaError_t launch_group_norm_bwd(const void* dy, const void* x, const float* w, const float* bias, const void* gate,
                                  void* dx, float* dw, float* dbias, void* dgate, int B, int L, int C, int G, float eps,
                                  int channel_major, int vec, float* part, int dtype, cudaStream_t st) {
  const NormArgs p{x, gate, dy, w, bias, (long long)B * L, L, C, G, C / G, eps, (float)(1.0 / (C / G)), vec};
  const Parts q = parts(B, L, C, G, channel_major);
  const int splits = q.count;
  cudaError_t e;
  switch (dtype) {
    case 0: e = bwd<float>(p, dx, dgate, part, splits, channel_major, st); break;
    case 1: e = bwd<__half>(p, dx, dgate, part, splits, channel_major, st); break;
    case 2: e = bwd<__nv_bfloat16>(p, dx, dgate, part, splits, channel_major, st); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  norm_sum_kernel<<<(2 * C + 7) / 8, 256, 0, st>>>(part, dw, dbias, C, C / G, G, q.groups, q.first, q.count);
  return cudaGetLastError();
}

}  // namespace fc
