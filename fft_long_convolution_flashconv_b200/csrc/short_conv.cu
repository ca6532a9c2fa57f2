// Short causal convolution by channels (depthwise, K <= 8 taps) with a bias
// and SiLU, the layer in front of a selective scan: prompts, training, single
// tokens.
//
//   c[t] = bias + sum_{j<K} w[j] x[t-j],  y[t] = silu(c[t]) or c[t]
//
// x at negative times comes from state_in (the last K - 1 inputs of the part
// before, oldest first) or is zero.  The floor is bytes: one read of x and one
// write of y (backward: x, dy, dx).  Measured in fp16 with four taps: 140 to 145 us for
// 1 x 2560 x 65536 (4.6 to 4.8 TB/s, issue slots 63% busy), 10 us forward and 26 us
// backward for 8 x 768 x 1024 (62 instructions an element at 51% of the issue slots:
// a thread's next loads wait for its arithmetic), 178 us backward for 8 x 768 x 8192.
#include "kernels.cuh"
#include "rows.cuh"

namespace fc {
namespace {

constexpr int kThreads = 128;

struct ConvArgs {
  Rows x, dy;
  const float* w;
  const float* bias;
  const int* lengths;
  const void* state_in;
  const void* dstate_out;
  int B, H, L, silu;
  int out_vec;
};

// x[t] for t < 0: the state entering the row.
template <typename T, int K>
__device__ __forceinline__ float past(const T* s, int t) {
  return s ? IO<T>::ldplain(s + (K - 1) + t) : 0.f;
}

// A thread computes kPer vectors of eight outputs of a row, a block's width apart.
// A vector and the one before it (from L1) hold every input it needs, K - 1 <= 7;
// all of a thread's loads are issued before the first is used.
constexpr int kPer = 4;

template <typename T, int K>
__global__ __launch_bounds__(kThreads) void short_conv_kernel(ConvArgs p, T* y, T* state_out, int nvec, int tx_log,
                                                              unsigned nblk_x) {
  const int tx = threadIdx.x & ((1 << tx_log) - 1), ty = threadIdx.x >> tx_log;
  const unsigned by = blockIdx.x / nblk_x, bx = blockIdx.x - by * nblk_x;
  const unsigned row = by * (kThreads >> tx_log) + ty;
  const int v0 = (int)(bx * kPer << tx_log) + tx;
  if (row >= (unsigned)p.B * p.H || v0 >= nvec) return;
  const unsigned b = row / p.H, h = row - b * p.H;
  const int n = row_length(p.lengths, b, p.L);
  const T* x = (const T*)p.x.p + b * p.x.bs + h * p.x.rs;
  const T* s = p.state_in ? (const T*)p.state_in + (long long)row * (K - 1) : nullptr;
  T* out = y + (long long)row * p.L;
  float w[K];
#pragma unroll
  for (int j = 0; j < K; ++j) w[j] = __ldg(p.w + (long long)h * K + j);
  const float bias = p.bias ? __ldg(p.bias + h) : 0.f;
  auto outputs = [&](int t0, const float (&a)[16]) {  // a: x[t0 - 8 .. t0 + 7]
    float o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 c = both(bias);
#pragma unroll
      for (int j = 0; j < K; ++j) {
        c.x = fmaf(w[j], a[8 + 2 * i - j], c.x);
        c.y = fmaf(w[j], a[9 + 2 * i - j], c.y);
      }
      if (p.silu) c = silu2(c);
      o[2 * i] = c.x;
      o[2 * i + 1] = c.y;
    }
    store8(out, t0, p.L, n, p.out_vec, o);
  };
  auto before = [&](float (&v)[8]) {  // the inputs before the row
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i >= 9 - K ? past<T, K>(s, i - 8) : 0.f;
  };
  const int last = v0 + ((kPer - 1) << tx_log);
  if (p.x.vec && (last + 1) * 8 <= n) {  // whole vectors inside the row
    Raw8<T> own[kPer], prev[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const T* q = x + (v0 + (j << tx_log)) * 8;
      ldraw8(q, own[j]);
      if (K > 1 && (j > 0 || v0 > 0)) ldraw8(q - 8, prev[j]);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      float v[8], a[16];
      if (K > 1) {
        unpack8(prev[j], v);
        if (j == 0 && v0 == 0) before(v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = v[i];
      unpack8(own[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[8 + i] = v[i];
      outputs((v0 + (j << tx_log)) * 8, a);
    }
  } else {
    for (int vec = v0; vec <= last && vec < nvec; vec += 1 << tx_log) {
      const int t0 = vec * 8;
      float v[8], a[16];
      if (t0 > 0)
        load8(x, t0 - 8, p.L, n, p.x.vec, v);
      else
        before(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = v[i];
      load8(x, t0, p.L, n, p.x.vec, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[8 + i] = v[i];
      outputs(t0, a);
    }
  }
  if (state_out && v0 == 0) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      const int t = n - (K - 1) + i;
      IO<T>::st(state_out + (long long)row * (K - 1) + i, t >= 0 ? IO<T>::ldplain(x + t) : past<T, K>(s, t));
    }
  }
}

// Backward.  dc[t] = dy[t] silu'(c[t]);
//   dx[t] = sum_j w[j] dc[t+j] (+ dstate_out),  dw[j] = sum_{b,t} dc[t] x[t-j],  dbias = sum dc.
// A block takes one channel and part of its (batch row, vector) items; a
// thread recomputes the K - 1 values of c behind its vector instead of
// waiting for its neighbour's.  dw and dbias are summed in registers, then
// over the block in a fixed order into part[split][h][K + 1].
template <typename T, int K>
__global__ __launch_bounds__(kThreads) void short_conv_bwd_kernel(ConvArgs p, T* dx, T* dstate_in, float* part,
                                                                  float* dw_out, float* db_out, int nvec,
                                                                  int per_split) {
  const int h = blockIdx.x;
  const long long items = (long long)p.B * nvec;
  const long long lo = (long long)blockIdx.y * per_split;
  const int count = (int)(lo + per_split < items ? per_split : items - lo);  // may be below 1
  float w[K], dw[K], db = 0.f;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    w[j] = __ldg(p.w + (long long)h * K + j);
    dw[j] = 0.f;
  }
  const float bias = p.bias ? __ldg(p.bias + h) : 0.f;
  // item lo + i of the channel: batch row b, vector vec
  int b = (int)((lo + threadIdx.x) / nvec), vec = (int)((lo + threadIdx.x) % nvec);
  const int db_step = kThreads / nvec, dv_step = kThreads % nvec;
  for (int i0 = threadIdx.x; i0 < count; i0 += kThreads) {
    const int t0 = vec * 8;
    const long long row = (long long)b * p.H + h;
    const int n = row_length(p.lengths, b, p.L);
    const T* x = (const T*)p.x.p + b * p.x.bs + h * p.x.rs;
    const T* dy = (const T*)p.dy.p + b * p.dy.bs + h * p.dy.rs;
    const T* s = p.state_in ? (const T*)p.state_in + row * (K - 1) : nullptr;
    const T* ds = p.dstate_out ? (const T*)p.dstate_out + row * (K - 1) : nullptr;
    float a[24], dc[16];
    {
      float v[8];
      if (t0 > 0) {
        load8(x, t0 - 8, p.L, n, p.x.vec, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i >= 9 - K ? past<T, K>(s, i - 8) : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = v[i];
      load8(x, t0, p.L, n, p.x.vec, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) a[8 + i] = v[i];
      load8(dy, t0, p.L, n, p.dy.vec, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) dc[i] = v[i];
      if (K > 1 && t0 + 8 < n) {
        load8(x, t0 + 8, p.L, n, p.x.vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) a[16 + i] = v[i];
        load8(dy, t0 + 8, p.L, n, p.dy.vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) dc[8 + i] = v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) a[16 + i] = dc[8 + i] = 0.f;
      }
    }
    const bool inner = t0 + 7 + K <= n;  // everything below lies in the row
    if (p.silu) {
#pragma unroll
      for (int i = 0; i < 8 + K; i += 2) {  // pairs; the last may be one too many
        float2 c = both(bias);
#pragma unroll
        for (int j = 0; j < K; ++j) {
          c.x = fmaf(w[j], a[8 + i - j], c.x);
          if (i + 1 < 16) c.y = fmaf(w[j], a[9 + i - j], c.y);
        }
        c = dsilu2(c);
        dc[i] *= c.x;
        if (i + 1 < 16) dc[i + 1] *= c.y;
      }
    }
    if (!inner) {  // a zero gradient behind the row's end stays one whatever c was
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (t0 + i >= n) dc[i] = 0.f;
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < K; ++j) v = fmaf(w[j], dc[i + j], v);
      o[i] = v;
    }
    if (inner) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        db += dc[i];
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j] = fmaf(dc[i], a[8 + i - j], dw[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int k = t0 + i - (n - (K - 1));  // this input's place in state_out
        if (ds && k >= 0 && k < K - 1) o[i] += IO<T>::ldplain(ds + k);
        if (t0 + i >= n) continue;
        db += dc[i];
#pragma unroll
        for (int j = 0; j < K; ++j) dw[j] = fmaf(dc[i], a[8 + i - j], dw[j]);
      }
    }
    store8(dx + row * p.L, t0, p.L, n, p.out_vec, o);
    if (dstate_in && vec == 0) {
#pragma unroll
      for (int i = 0; i < K - 1; ++i) {  // x at time i - (K - 1)
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < K; ++j) {
          const int t = i - (K - 1) + j;
          if (t >= 0) v = fmaf(w[j], dc[t], v);
        }
        const int k = i - n;  // where the same input stands in state_out
        if (ds && k >= 0) v += IO<T>::ldplain(ds + k);
        IO<T>::st(dstate_in + row * (K - 1) + i, v);
      }
    }
    b += db_step;
    vec += dv_step;
    if (vec >= nvec) {
      vec -= nvec;
      ++b;
    }
  }
  // sums over the block, in a fixed order
  __shared__ float red[kThreads / 32][K + 1];
#pragma unroll
  for (int j = 0; j <= K; ++j) {
    float v = j < K ? dw[j < K ? j : 0] : db;
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(~0u, v, d);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5][j] = v;
  }
  __syncthreads();
  if (threadIdx.x <= K) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) v += red[i][threadIdx.x];
    if (gridDim.y > 1)
      part[((long long)blockIdx.y * p.H + h) * (K + 1) + threadIdx.x] = v;
    else if (threadIdx.x < K)
      dw_out[(long long)h * K + threadIdx.x] = v;
    else if (db_out)
      db_out[h] = v;
  }
}

// dw and dbias from the splits' parts, in order.
__global__ void short_conv_sum_kernel(const float* part, float* dw, float* dbias, int H, int K, int splits) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long m = (long long)H * (K + 1);
  if (i >= m) return;
  float v = 0.f;
  for (int s = 0; s < splits; ++s) v += part[s * m + i];
  const long long h = i / (K + 1);
  const int j = (int)(i % (K + 1));
  if (j < K)
    dw[h * K + j] = v;
  else if (dbias)
    dbias[h] = v;
}

// One token: the window is the state and the new input; the state moves on by one.
template <typename T, int K>
__global__ __launch_bounds__(kThreads) void short_conv_step_kernel(const T* x, long long xs, T* state, const float* w,
                                                                   const float* bias, T* y, int H, int silu_on,
                                                                   const int* slots, int S) {
  const int b = blockIdx.y, h = blockIdx.x * kThreads + threadIdx.x;
  const int slot = batch_slot(slots, b, S);
  if (h >= H) return;
  if (slot < 0) {
    IO<T>::st(y + (long long)b * H + h, 0.f);
    return;
  }
  T* s = state + ((long long)slot * H + h) * (K - 1);
  const T xn = x[b * xs + h];
  float c = bias ? __ldg(bias + h) : 0.f;
  T win[K];
#pragma unroll
  for (int i = 0; i < K - 1; ++i) win[i] = s[i];
  win[K - 1] = xn;
#pragma unroll
  for (int j = 0; j < K; ++j) c = fmaf(__ldg(w + (long long)h * K + j), IO<T>::ldplain(&win[K - 1 - j]), c);
#pragma unroll
  for (int i = 0; i < K - 1; ++i) s[i] = win[i + 1];
  IO<T>::st(y + (long long)b * H + h, silu_on ? silu(c) : c);
}

template <typename T, int K>
cudaError_t fwd(const ConvArgs& p, void* y, void* state_out, cudaStream_t st) {
  const int nvec = (p.L + 7) / 8;
  int tx_log = 0;  // threads along a row: shorter rows share a block
  while ((1 << tx_log) < kThreads && (kPer << tx_log) < nvec) ++tx_log;
  const long long rows = (long long)p.B * p.H, rpb = kThreads >> tx_log, wide = (long long)kPer << tx_log;
  const long long nblk_x = (nvec + wide - 1) / wide;
  const long long grid = (rows + rpb - 1) / rpb * nblk_x;
  short_conv_kernel<T, K><<<(unsigned)grid, kThreads, 0, st>>>(p, (T*)y, (T*)state_out, nvec, tx_log,
                                                               (unsigned)nblk_x);
  return cudaGetLastError();
}

template <typename T, int K>
cudaError_t bwd(const ConvArgs& p, void* dx, float* dw, float* dbias, void* dstate_in, float* part, int splits,
                cudaStream_t st) {
  const int nvec = (p.L + 7) / 8;
  const long long items = (long long)p.B * nvec;
  const int per = (int)((items + splits - 1) / splits);
  short_conv_bwd_kernel<T, K><<<dim3(p.H, splits), kThreads, 0, st>>>(p, (T*)dx, (T*)dstate_in, part, dw, dbias, nvec,
                                                                     per);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  const long long m = (long long)p.H * (K + 1);
  short_conv_sum_kernel<<<(unsigned)((m + 255) / 256), 256, 0, st>>>(part, dw, dbias, p.H, K, splits);
  return cudaGetLastError();
}

template <typename T, int K>
cudaError_t step(const void* x, long long xs, void* state, const float* w, const float* bias, void* y, int B, int H,
                 int silu, const int* slots, int S, cudaStream_t st) {
  short_conv_step_kernel<T, K><<<dim3((H + kThreads - 1) / kThreads, B), kThreads, 0, st>>>(
      (const T*)x, xs, (T*)state, w, bias, (T*)y, H, silu, slots, S);
  return cudaGetLastError();
}

// f.template operator()<T, K>() for the runtime type and number of taps
template <typename T, typename F>
cudaError_t by_taps(int K, F f) {
  switch (K) {
    case 1: return f.template operator()<T, 1>();
    case 2: return f.template operator()<T, 2>();
    case 3: return f.template operator()<T, 3>();
    case 4: return f.template operator()<T, 4>();
    case 5: return f.template operator()<T, 5>();
    case 6: return f.template operator()<T, 6>();
    case 7: return f.template operator()<T, 7>();
    case 8: return f.template operator()<T, 8>();
    default: return cudaErrorInvalidValue;
  }
}
template <typename F>
cudaError_t by_type(int dtype, int K, F f) {
  switch (dtype) {
    case 0: return by_taps<float>(K, f);
    case 1: return by_taps<__half>(K, f);
    case 2: return by_taps<__nv_bfloat16>(K, f);
    default: return cudaErrorInvalidValue;
  }
}

struct FwdCall {
  const ConvArgs& p;
  void *y, *state_out;
  cudaStream_t st;
  template <typename T, int K> cudaError_t operator()() const { return fwd<T, K>(p, y, state_out, st); }
};
struct BwdCall {
  const ConvArgs& p;
  void* dx;
  float *dw, *dbias;
  void* dstate_in;
  float* part;
  int splits;
  cudaStream_t st;
  template <typename T, int K> cudaError_t operator()() const {
    return bwd<T, K>(p, dx, dw, dbias, dstate_in, part, splits, st);
  }
};
struct StepCall {
  const void* x;
  long long xs;
  void* state;
  const float *w, *bias;
  void* y;
  int B, H, silu;
  const int* slots;
  int S;
  cudaStream_t st;
  template <typename T, int K> cudaError_t operator()() const {
    return step<T, K>(x, xs, state, w, bias, y, B, H, silu, slots, S, st);
  }
};

}  // namespace

cudaError_t launch_short_conv(const Rows& x, const float* w, const float* bias, void* y, int B, int H, int L, int K,
                              int silu, const int* lengths, const void* state_in, void* state_out, int out_vec,
                              int dtype, cudaStream_t st) {
  const ConvArgs p{x, Rows{}, w, bias, lengths, state_in, nullptr, B, H, L, silu, out_vec};
  return by_type(dtype, K, FwdCall{p, y, state_out, st});
}

// Parts of dw and dbias over the (batch row, vector) items of a channel: enough
// blocks for each of 148 SMs to hold four (592), each thread with at least one item.
// (A number, not the device's count: the workspace's size is the same everywhere.)  One part
// needs no second kernel: at 8 x 768 channels of 1024 steps in fp16, forward and
// backward together take 28 us either way, and the call 22 us of the host's time
// instead of 27.  Longer rows were not measured with more parts.
int short_conv_bwd_splits(int B, int H, int L) {
  const long long items = (long long)B * ((L + 7) / 8);
  const long long most = (items + kThreads - 1) / kThreads;
  long long s = (592 + H - 1) / H;
  const long long least = (items + (1 << 30) - 1) >> 30;  // items of a split are counted in an int
  if (s > most) s = most;
  if (s < least) s = least;
  return (int)(s < 1 ? 1 : s);
}

cudaError_t launch_short_conv_bwd(const Rows& dy, const Rows& x, const float* w, const float* bias, void* dx, float* dw,
                                  float* dbias, int B, int H, int L, int K, int silu, const int* lengths,
                                  const void* state_in, const void* dstate_out, void* dstate_in, float* part,
                                  int out_vec, int dtype, cudaStream_t st) {
  const ConvArgs p{x, dy, w, bias, lengths, state_in, dstate_out, B, H, L, silu, out_vec};
  return by_type(dtype, K, BwdCall{p, dx, dw, dbias, dstate_in, part, short_conv_bwd_splits(B, H, L), st});
}

cudaError_t launch_short_conv_step(const void* x, long long xs, void* state, const float* w, const float* bias, void* y,
                                   int B, int H, int K, int silu, const int* slots, int S, int dtype,
                                   cudaStream_t st) {
  return by_type(dtype, K, StepCall{x, xs, state, w, bias, y, B, H, silu, slots, S, st});
}

}  // namespace fc
