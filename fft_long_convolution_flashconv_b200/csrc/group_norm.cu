// Group norm of each token on its own (so a causal model stays causal) with
// SiLU: what a mixer's output goes through, one group a head.
//
//   xh = (x - mean) rstd over the C / G channels of a group of one token
//   n = xh w + bias,  y = silu(n), or n silu(gate) with a gate
//
// x and gate are B x L x C (a mixer's output) or B x C x L (a scan's output);
// y is B x L x C for the output projection.  Bound by bytes: every kernel
// reads each input once, keeps a group's values in registers for the mean, the
// sum of squares around it and the output, and writes once.
#include "kernels.cuh"
#include "rows.cuh"

namespace fc {
namespace {

constexpr int kThreads = 256;

struct NormArgs {
  const void *x, *gate, *dy;
  const float *w, *bias;
  long long tokens;  // B * L
  int L, C, G, M;    // M = C / G
  float eps;
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

template <bool BLOCK, int V>
__device__ __forceinline__ void stats(float (&x)[V][8], int lane, int P, int M, float eps, float* red, float& mean,
                                      float& rstd) {
  float s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) s += x[v][i];
  mean = sum_unit<BLOCK>(s, P, red) / M;
  s = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((v * P + lane) * 8 + i < M) s = fmaf(x[v][i] - mean, x[v][i] - mean, s);
  rstd = rsqrtf(sum_unit<BLOCK>(s, P, red) / M + eps);
}

// P lanes (or the block) share a group of one token, V vectors of eight channels each.
template <typename T, int V, bool BLOCK>
__global__ __launch_bounds__(kThreads) void norm_kernel(NormArgs p, T* y, int P) {
  __shared__ float red[kThreads / 32];
  const int lane = threadIdx.x % P;
  const long long units = p.tokens * p.G;
  const long long unit0 = (long long)blockIdx.x * (kThreads / P) + threadIdx.x / P;
  const bool live = unit0 < units;
  const long long unit = live ? unit0 : 0;
  const int g = (int)(unit % p.G), M = p.M;
  const T* x = (const T*)p.x + unit * M;
  float xv[V][8], mean, rstd;
#pragma unroll
  for (int v = 0; v < V; ++v) ld_group(x, (v * P + lane) * 8, M, p.vec, xv[v]);
  stats<BLOCK, V>(xv, lane, P, M, p.eps, red, mean, rstd);
  if (!live) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int m = (v * P + lane) * 8;
    float w[8], bias[8], o[8];
    ld_param(p.w ? p.w + (long long)g * M : nullptr, m, M, 1.f, w);
    ld_param(p.bias ? p.bias + (long long)g * M : nullptr, m, M, 0.f, bias);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf((xv[v][i] - mean) * rstd, w[i], bias[i]);
    if (p.gate) {
      float z[8];
      ld_group((const T*)p.gate + unit * M, m, M, p.vec, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= silu(z[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = silu(o[i]);
    }
    st_group(y + unit * M, m, M, p.vec, o);
  }
}

// Backward.  dn = dy silu'(n) (dy silu(gate) with a gate), e = dn w,
//   dx = rstd (e - mean(e) - xh mean(e xh)),  dw = sum dn xh,  dbias = sum dn.
// A block takes one group and part of the tokens, so that a lane keeps its
// channels' dw and dbias in registers; the parts are joined in a fixed order.
template <typename T, int V, bool BLOCK>
__global__ __launch_bounds__(kThreads) void norm_bwd_kernel(NormArgs p, T* dx, T* dgate, float* part, int P,
                                                            long long per_split) {
  __shared__ float red[kThreads / 32];
  __shared__ float acc[kThreads * 8 * V];
  const int lane = threadIdx.x % P, sub = threadIdx.x / P, subs = kThreads / P, g = blockIdx.x, M = p.M;
  const long long lo = blockIdx.y * per_split, hi = lo + per_split < p.tokens ? lo + per_split : p.tokens;
  float dw[V][8] = {}, db[V][8] = {};
  for (long long base = lo; base < hi; base += subs) {
    const bool live = base + sub < hi;
    const long long off = ((live ? base + sub : lo) * p.G + g) * M;
    float x[V][8], dn[V][8], mean, rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ld_group((const T*)p.x + off, (v * P + lane) * 8, M, p.vec, x[v]);
      ld_group((const T*)p.dy + off, (v * P + lane) * 8, live ? M : 0, p.vec, dn[v]);
    }
    stats<BLOCK, V>(x, lane, P, M, p.eps, red, mean, rstd);
    float se = 0.f, sex = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int m = (v * P + lane) * 8;
      float w[8], bias[8];
      ld_param(p.w ? p.w + (long long)g * M : nullptr, m, M, 1.f, w);
      ld_param(p.bias ? p.bias + (long long)g * M : nullptr, m, M, 0.f, bias);
      float z[8], dg[8];
      if (p.gate) ld_group((const T*)p.gate + off, m, M, p.vec, z);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[v][i] = m + i < M ? (x[v][i] - mean) * rstd : 0.f;  // xh from here on
        const float n = fmaf(x[v][i], w[i], bias[i]);
        if (p.gate) {
          dg[i] = dn[v][i] * n * dsilu(z[i]);
          dn[v][i] *= silu(z[i]);
        } else {
          dn[v][i] *= dsilu(n);
        }
        dw[v][i] = fmaf(dn[v][i], x[v][i], dw[v][i]);
        db[v][i] += dn[v][i];
        dn[v][i] *= w[i];  // e from here on
        se += dn[v][i];
        sex = fmaf(dn[v][i], x[v][i], sex);
      }
      if (p.gate && live) st_group(dgate + off, m, M, p.vec, dg);
    }
    se = sum_unit<BLOCK>(se, P, red) / M;
    sex = sum_unit<BLOCK>(sex, P, red) / M;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = rstd * (dn[v][i] - se - x[v][i] * sex);
      if (live) st_group(dx + off, (v * P + lane) * 8, M, p.vec, o);
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[sub * (P * 8 * V) + (v * P + lane) * 8 + i] = which ? db[v][i] : dw[v][i];
    __syncthreads();
    for (int m = threadIdx.x; m < M; m += kThreads) {
      float s = 0.f;
      for (int k = 0; k < subs; ++k) s += acc[k * (P * 8 * V) + m];
      part[((long long)blockIdx.y * 2 + which) * p.C + (long long)g * M + m] = s;
    }
  }
}

__global__ void norm_sum_kernel(const float* part, float* dw, float* dbias, int C, int splits) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= 2 * C) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += part[(long long)s * 2 * C + i];
  if (i < C) {
    if (dw) dw[i] = v;
  } else if (dbias) {
    dbias[i - C] = v;
  }
}

// ------------------------------------------------------------------ B x C x L
// A block takes 64 tokens of a group.  A thread holds eight tokens (one 16-byte
// access of a channel's row) of every 32nd channel, V at a time; sums over the
// channels go over shuffles and shared memory.  Token-major rows (y, dy) pass
// through a shared tile of 64 tokens by 32 V channels whose vectors of eight
// channels are swizzled by the token, so that both directions of the
// transposition touch all banks.
constexpr int TT = 64;

template <int V>
__device__ __forceinline__ int tile_pos(int t, int m) {  // row of at least 64 channels: eight vectors
  constexpr int W = 32 * V < 64 ? 64 : 32 * V;
  return t * W + ((((m >> 3) & ~7) | (((m >> 3) ^ (t >> 3)) & 7)) << 3) + (m & 7);
}
template <int V> constexpr size_t tile_elems() { return (size_t)TT * (32 * V < 64 ? 64 : 32 * V); }

// Sums over all 32 channel threads of the eight tokens that a thread holds.
__device__ __forceinline__ void sum_tokens(float (&s)[8], float (*red)[TT]) {
  const int tv = threadIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] += __shfl_xor_sync(~0u, s[i], 8);
    s[i] += __shfl_xor_sync(~0u, s[i], 16);
  }
  __syncthreads();
  if (lane < 8)
#pragma unroll
    for (int i = 0; i < 8; ++i) red[warp][tv * 8 + i] = s[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] += red[w][tv * 8 + i];
}

template <typename T, int V>
struct Slab {  // the rows of a group that a block works on
  const NormArgs& p;
  long long row0;  // of the group's first channel
  int t0;          // first token of the thread
  __device__ __forceinline__ void load(const void* a, int m0, float (&v)[V][8]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int m = m0 + 32 * j + (threadIdx.x >> 3);
      load8((const T*)a + (row0 + (m < p.M ? m : 0)) * p.L, t0, p.L, m < p.M ? p.L : 0, p.vec, v[j]);
    }
  }
  __device__ __forceinline__ void store(void* a, int m, float (&v)[8]) const {
    if (m < p.M && t0 < p.L) store8((T*)a + (row0 + m) * p.L, t0, p.L, p.L, p.vec, v);
  }
};

// Mean and rstd of the thread's eight tokens; x holds the slab on return where there is only one.
template <typename T, int V>
__device__ __forceinline__ void stats_cm(const Slab<T, V>& sl, int M, float eps, float (&x)[V][8], float (*red)[TT],
                                         float (&mean)[8], float (&rstd)[8]) {
  const int mq = threadIdx.x >> 3;
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
  for (int i = 0; i < 8; ++i) mean[i] /= M;
  for (int m0 = 0; m0 < M; m0 += 32 * V) {
    if (M > 32 * V) sl.load(sl.p.x, m0, x);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (m0 + 32 * j + mq < M)
#pragma unroll
        for (int i = 0; i < 8; ++i) rstd[i] = fmaf(x[j][i] - mean[i], x[j][i] - mean[i], rstd[i]);
  }
  sum_tokens(rstd, red);
#pragma unroll
  for (int i = 0; i < 8; ++i) rstd[i] = rsqrtf(rstd[i] / M + eps);
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void norm_cm_kernel(NormArgs p, T* y, int tiles) {
  extern __shared__ float4 smem4[];
  T* tile = reinterpret_cast<T*>(smem4);
  __shared__ float red[kThreads / 32][TT];
  const int tl = blockIdx.x % tiles;
  const long long bg = blockIdx.x / tiles, b = bg / p.G;
  const int g = (int)(bg % p.G), M = p.M, tv = threadIdx.x & 7, mq = threadIdx.x >> 3, tb = tl * TT;
  const Slab<T, V> sl{p, b * p.C + (long long)g * M, tb + tv * 8};
  float x[V][8], mean[8], rstd[8];
  stats_cm<T, V>(sl, M, p.eps, x, red, mean, rstd);
  for (int m0 = 0; m0 < M; m0 += 32 * V) {
    if (M > 32 * V) sl.load(p.x, m0, x);
    float z[V][8];
    if (p.gate) sl.load(p.gate, m0, z);
    __syncthreads();  // the tile may still be read
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int mm = 32 * j + mq, m = m0 + mm;
      if (m >= M) continue;
      const float w = p.w ? __ldg(p.w + (long long)g * M + m) : 1.f;
      const float bias = p.bias ? __ldg(p.bias + (long long)g * M + m) : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = fmaf((x[j][i] - mean[i]) * rstd[i], w, bias);
        IO<T>::st(tile + tile_pos<V>(tv * 8 + i, mm), p.gate ? n * silu(z[j][i]) : silu(n));
      }
    }
    __syncthreads();
    const int width = min(32 * V, M - m0), chunks = (width + 7) / 8;
    for (int k = threadIdx.x; k < TT * chunks; k += kThreads) {
      const int t = k / chunks, mm = k % chunks * 8;
      if (tb + t >= p.L) break;
      T* o = y + (b * p.L + tb + t) * p.C + (long long)g * M + m0 + mm;
      const T* s = tile + tile_pos<V>(t, mm);
      if (mm + 8 <= width && ((uintptr_t)o & 15) == 0) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4*>(o)[i] = reinterpret_cast<const uint4*>(s)[i];
      } else {
        for (int i = 0; i < 8 && mm + i < width; ++i) o[i] = s[i];
      }
    }
  }
}

template <typename T, int V>
__global__ __launch_bounds__(kThreads) void norm_cm_bwd_kernel(NormArgs p, T* dx, T* dgate, float* part, int tiles,
                                                               int per_split) {
  extern __shared__ float4 smem4[];
  float* acc = reinterpret_cast<float*>(smem4);  // [2][M] dw, dbias of the block
  const int Ma = (p.M + 3) / 4 * 4;
  T* tile = reinterpret_cast<T*>(acc + 2 * Ma);
  __shared__ float red[kThreads / 32][TT];
  const int g = blockIdx.x, M = p.M, tv = threadIdx.x & 7, mq = threadIdx.x >> 3;
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
        const int width = min(32 * V, M - m0), chunks = (width + 7) / 8;
        if (M > 32 * V || pass == 0) {  // dy of the slab into the tile
          __syncthreads();
          for (int k = threadIdx.x; k < TT * chunks; k += kThreads) {
            const int t = k / chunks, mm = k % chunks * 8;
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
          }
          __syncthreads();
        }
        if (M > 32 * V) sl.load(p.x, m0, x);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int mm = 32 * j + mq, m = m0 + mm;
          const bool ok = m < M;
          const float w = ok && p.w ? __ldg(p.w + (long long)g * M + m) : 1.f;
          const float bias = ok && p.bias ? __ldg(p.bias + (long long)g * M + m) : 0.f;
          float z[8], o[8], dg[8], sw = 0.f, sb = 0.f;
          if (p.gate)
            load8((const T*)p.gate + (sl.row0 + (ok ? m : 0)) * p.L, sl.t0, p.L, ok ? p.L : 0, p.vec, z);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float xh = (x[j][i] - mean[i]) * rstd[i];
            const float dy = ok ? IO<T>::ldplain(tile + tile_pos<V>(tv * 8 + i, mm)) : 0.f;
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
          se[i] /= M;
          sex[i] /= M;
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

template <typename T, int V, bool BLOCK>
cudaError_t fwd_v(const NormArgs& p, void* y, int P, cudaStream_t st) {
  const long long units = p.tokens * p.G, per = kThreads / P;
  norm_kernel<T, V, BLOCK><<<(unsigned)((units + per - 1) / per), kThreads, 0, st>>>(p, (T*)y, P);
  return cudaGetLastError();
}
template <typename T, int V, bool BLOCK>
cudaError_t bwd_v(const NormArgs& p, void* dx, void* dgate, float* part, int P, int splits, cudaStream_t st) {
  const long long per = (p.tokens + splits - 1) / splits;
  norm_bwd_kernel<T, V, BLOCK><<<dim3(p.G, splits), kThreads, 0, st>>>(p, (T*)dx, (T*)dgate, part, P, per);
  return cudaGetLastError();
}
template <typename T, int V>
cudaError_t fwd_cm(const NormArgs& p, void* y, cudaStream_t st) {
  const int tiles = (p.L + TT - 1) / TT;
  const size_t smem = tile_elems<V>() * sizeof(T);
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
  const NormArgs p{x, gate, nullptr, w, bias, (long long)B * L, L, C, G, C / G, eps, vec};
  switch (dtype) {
    case 0: return fwd<float>(p, y, channel_major, st);
    case 1: return fwd<__half>(p, y, channel_major, st);
    case 2: return fwd<__nv_bfloat16>(p, y, channel_major, st);
    default: return cudaErrorInvalidValue;
  }
}

// Parts of the tokens: about eight blocks an SM, each with a few tokens for every group of lanes.
int group_norm_bwd_splits(int B, int L, int C, int G, int channel_major) {
  const Plan r = plan(C / G);
  const long long items = channel_major ? (long long)B * ((L + TT - 1) / TT)
                                        : ((long long)B * L + 4 * (kThreads / r.P) - 1) / (4 * (kThreads / r.P));
  long long s = (1184 + G - 1) / G;
  if (s > items) s = items;
  return (int)(s < 1 ? 1 : s);
}

cudaError_t launch_group_norm_bwd(const void* dy, const void* x, const float* w, const float* bias, const void* gate,
                                  void* dx, float* dw, float* dbias, void* dgate, int B, int L, int C, int G, float eps,
                                  int channel_major, int vec, float* part, int dtype, cudaStream_t st) {
  const NormArgs p{x, gate, dy, w, bias, (long long)B * L, L, C, G, C / G, eps, vec};
  const int splits = group_norm_bwd_splits(B, L, C, G, channel_major);
  cudaError_t e;
  switch (dtype) {
    case 0: e = bwd<float>(p, dx, dgate, part, splits, channel_major, st); break;
    case 1: e = bwd<__half>(p, dx, dgate, part, splits, channel_major, st); break;
    case 2: e = bwd<__nv_bfloat16>(p, dx, dgate, part, splits, channel_major, st); break;
    default: return cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  norm_sum_kernel<<<(2 * C + 255) / 256, 256, 0, st>>>(part, dw, dbias, C, splits);
  return cudaGetLastError();
}

}  // namespace fc
