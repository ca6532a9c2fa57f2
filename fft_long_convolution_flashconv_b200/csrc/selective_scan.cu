// Selective scan: the diagonal SSM whose step size, input and output vectors
// depend on the input, for prompts and for single tokens.
//
//   dt = softplus(delta + dt_bias),  a_n = exp(dt A_n)
//   x_n <- a_n x_n + dt B_n u,  y = (sum_n C_n x_n + D u) silu(z)
//
// A lane holds eight steps of one channel in registers and runs through the
// states one after the other: it forms a_n and dt B_n u for its steps, runs
// the recurrence from zero, joins the lanes of a channel by a scan of (product
// of a, end state) over shuffles, runs the recurrence again from the state
// that enters it and adds C_n x_n to its eight outputs.  The product of a over
// a lane is exp(A_n sum dt), one exponential.  TL lanes are a channel's
// TL * 8 steps, so global rows are read in 16-byte vectors of neighbouring
// lanes; a block's channels share B and C through shared memory.
#include "kernels.cuh"
#include "scan.cuh"

namespace fc {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStates = 16;  // states whose B and C are in shared memory at a time

template <typename T, int TL>
__global__ __launch_bounds__(kThreads) void scan_kernel(ScanArgs p, T* y, float* state_out, float* ckpt, int tiles) {
  constexpr int CL = 32 / TL, TB = TL * 8, CH = kWarps * CL;
  extern __shared__ float4 smem4[];
  float* Bs = reinterpret_cast<float*>(smem4);  // [kStates][TB]
  float* Cs = Bs + kStates * TB;
  float* As = Cs + kStates * TB;  // [N][CH], A log2(e)
  float* xs = As + p.N * CH;      // [N][CH], the state entering the block of steps
  const int tid = threadIdx.x, lane = tid & 31, tl = lane % TL;
  const int c = (tid >> 5) * CL + lane / TL;  // channel of the block
  const int E = p.H / p.G;
  const int tile = blockIdx.x % tiles, bg = blockIdx.x / tiles, b = bg / p.G, g = bg % p.G;
  const bool live = tile * CH + c < E;
  const int h = g * E + (live ? tile * CH + c : 0);
  const long long row = (long long)b * p.H + h;
  const int n = row_length(p.lengths, b, p.L);
  const int N = p.N;
  for (int i = tid; i < N * CH; i += kThreads) {
    const int s = i / CH, cc = i % CH, hh = g * E + tile * CH + cc;
    const bool ok = tile * CH + cc < E;
    As[i] = ok ? __ldg(p.A + (long long)hh * N + s) * kLog2e : 0.f;
    xs[i] = ok && p.state_in ? __ldg(p.state_in + ((long long)b * p.H + hh) * N + s) : 0.f;
  }
  const T* u = (const T*)p.u.p + b * p.u.bs + h * p.u.rs;
  const T* delta = (const T*)p.delta.p + b * p.delta.bs + h * p.delta.rs;
  const T* z = p.z.p ? (const T*)p.z.p + b * p.z.bs + h * p.z.rs : nullptr;
  const T* Bt = (const T*)p.Bt.p + b * p.Bt.bs + g * p.Bt.gs;
  const T* Ct = (const T*)p.Ct.p + b * p.Ct.bs + g * p.Ct.gs;
  const float Dh = p.D ? __ldg(p.D + h) : 0.f, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
  const int nck = (p.L + kCkptSteps - 1) / kCkptSteps;
  for (int tb = 0; tb < p.L; tb += TB) {
    const int t0 = tb + tl * 8;
    float v[8], dt[8], du[8], o[8];
    if (tb < n) {
      load8(u, t0, p.L, n, p.u.vec, v);
      load8(delta, t0, p.L, n, p.delta.vec, dt);
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float r = dt[i] + bias;
        dt[i] = t0 + i < n ? (p.softplus ? softplus(r) : r) : 0.f;  // dt = 0 keeps the state
        sum += dt[i];
        du[i] = dt[i] * v[i];
        o[i] = Dh * v[i];
      }
      for (int s0 = 0; s0 < N; s0 += kStates) {
        const int ns = min(kStates, N - s0);
        __syncthreads();
        for (int i = tid; i < ns * TL; i += kThreads) {
          const int s = i / TL, k = i % TL;
          float w[8];
          load8(Bt + (long long)(s0 + s) * p.Bt.rs, tb + k * 8, p.L, n, p.Bt.vec, w);
          float4* d = reinterpret_cast<float4*>(Bs + s * TB);
          d[k] = make_float4(w[0], w[1], w[2], w[3]);
          d[TL + k] = make_float4(w[4], w[5], w[6], w[7]);
          load8(Ct + (long long)(s0 + s) * p.Ct.rs, tb + k * 8, p.L, n, p.Ct.vec, w);
          d = reinterpret_cast<float4*>(Cs + s * TB);
          d[k] = make_float4(w[0], w[1], w[2], w[3]);
          d[TL + k] = make_float4(w[4], w[5], w[6], w[7]);
        }
        __syncthreads();
#pragma unroll 2
        for (int s = 0; s < ns; ++s) {
          const float A2 = As[(s0 + s) * CH + c];
          const float4* Bp = reinterpret_cast<const float4*>(Bs + s * TB);
          const float4* Cp = reinterpret_cast<const float4*>(Cs + s * TB);
          const float4 b0 = Bp[tl], b1 = Bp[TL + tl];
          const float Bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
          float a[8], w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = ex2(dt[i] * A2);
            w[i] = du[i] * Bv[i];
          }
          float hh = w[0];
#pragma unroll
          for (int i = 1; i < 8; ++i) hh = fmaf(a[i], hh, w[i]);
          float P = ex2(sum * A2);
          float x0 = 0.f;
          if (tl == 0) {
            x0 = xs[(s0 + s) * CH + c];
            hh = fmaf(P, x0, hh);
          }
#pragma unroll
          for (int d = 1; d < TL; d *= 2) {  // state at the end of every lane
            const float hp = __shfl_up_sync(~0u, hh, d, TL);
            const float Pp = __shfl_up_sync(~0u, P, d, TL);
            if (tl >= d) {
              hh = fmaf(P, hp, hh);
              P *= Pp;
            }
          }
          const float up = __shfl_up_sync(~0u, hh, 1, TL);
          float x = tl == 0 ? x0 : up;
          __syncwarp();
          if (tl == TL - 1) xs[(s0 + s) * CH + c] = hh;
          if (ckpt && live && (t0 & (kCkptSteps - 1)) == 0 && t0 < n)
            ckpt[(row * nck + t0 / kCkptSteps) * N + s0 + s] = x;
          const float4 c0 = Cp[tl], c1 = Cp[TL + tl];
          const float Cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x = fmaf(a[i], x, w[i]);
            o[i] = fmaf(Cv[i], x, o[i]);
          }
        }
      }
      if (z) {
        float zv[8];
        load8(z, t0, p.L, n, p.z.vec, zv);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] *= silu(zv[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = 0.f;
    }
    if (live && t0 < p.L) store8(y + row * p.L, t0, p.L, n, p.out_vec, o);
  }
  if (state_out) {
    __syncthreads();
    for (int i = tid; i < N * CH; i += kThreads) {
      const int cc = i / N, s = i % N;
      if (tile * CH + cc < E) state_out[((long long)b * p.H + g * E + tile * CH + cc) * N + s] = xs[s * CH + cc];
    }
  }
}

// One token.  LPC lanes share a channel, each four states at a time (one
// 16-byte access where N is a multiple of four).
template <typename T>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(ScanArgs p, float* state, T* y, const int* slots, int S,
                                                             int lpc, int vec) {
  const int b = blockIdx.y, sub = threadIdx.x % lpc;
  const int h = blockIdx.x * (kThreads / lpc) + threadIdx.x / lpc;
  const int slot = batch_slot(slots, b, S);
  const bool live = h < p.H;
  const int hh = live ? h : 0, N = p.N, g = hh / (p.H / p.G);
  if (slot < 0) {
    if (live && sub == 0) IO<T>::st(y + (long long)b * p.H + h, 0.f);
    return;
  }
  const float u = IO<T>::ld((const T*)p.u.p + b * p.u.bs + hh * p.u.rs);
  float dt = IO<T>::ld((const T*)p.delta.p + b * p.delta.bs + hh * p.delta.rs);
  if (p.dt_bias) dt += __ldg(p.dt_bias + hh);
  if (p.softplus) dt = softplus(dt);
  const float du = dt * u;
  const T* Bt = (const T*)p.Bt.p + b * p.Bt.bs + g * p.Bt.gs;
  const T* Ct = (const T*)p.Ct.p + b * p.Ct.bs + g * p.Ct.gs;
  float* xp = state + ((long long)slot * p.H + hh) * N;
  const float* Ap = p.A + (long long)hh * N;
  float acc = 0.f;
  for (int s = sub * 4; s < N; s += lpc * 4) {
    float x[4], A[4];
    if (vec) {
      const float4 xv = *reinterpret_cast<const float4*>(xp + s), av = __ldg(reinterpret_cast<const float4*>(Ap + s));
      x[0] = xv.x; x[1] = xv.y; x[2] = xv.z; x[3] = xv.w;
      A[0] = av.x; A[1] = av.y; A[2] = av.z; A[3] = av.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = s + i < N ? xp[s + i] : 0.f;
        A[i] = s + i < N ? __ldg(Ap + s + i) : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (s + i >= N) break;
      x[i] = fmaf(ex2(dt * A[i] * kLog2e), x[i], du * IO<T>::ld(Bt + (s + i) * p.Bt.rs));
      acc = fmaf(IO<T>::ld(Ct + (s + i) * p.Ct.rs), x[i], acc);
    }
    if (live) {
      if (vec) {
        *reinterpret_cast<float4*>(xp + s) = make_float4(x[0], x[1], x[2], x[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (s + i < N) xp[s + i] = x[i];
      }
    }
  }
  for (int d = lpc / 2; d; d >>= 1) acc += __shfl_xor_sync(~0u, acc, d);
  if (live && sub == 0) {
    acc = fmaf(p.D ? __ldg(p.D + hh) : 0.f, u, acc);
    if (p.z.p) acc *= silu(IO<T>::ld((const T*)p.z.p + b * p.z.bs + hh * p.z.rs));
    IO<T>::st(y + (long long)b * p.H + h, acc);
  }
}

template <typename T, int TL>
cudaError_t run(const ScanArgs& p, void* y, float* state_out, float* ckpt, cudaStream_t st) {
  constexpr int CH = kWarps * 32 / TL, TB = TL * 8;
  const int tiles = (p.H / p.G + CH - 1) / CH;
  const size_t smem = (size_t)(2 * kStates * TB + 2 * p.N * CH) * 4;
  const cudaError_t e = smem_optin<scan_kernel<T, TL>>(smem);
  if (e != cudaSuccess) return e;
  scan_kernel<T, TL><<<(unsigned)((long long)tiles * p.B * p.G), kThreads, smem, st>>>(p, (T*)y, state_out, ckpt, tiles);
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const ScanArgs& p, void* y, float* state_out, float* ckpt, cudaStream_t st) {
  return run<T, 8>(p, y, state_out, ckpt, st);
}

template <typename T>
cudaError_t step(const ScanArgs& p, float* state, void* y, const int* slots, int S, cudaStream_t st) {
  int lpc = 1;
  while (lpc < 32 && lpc * 4 < p.N) lpc *= 2;
  const int per = kThreads / lpc;
  const int vec = p.N % 4 == 0 && ((uintptr_t)state & 15) == 0 && ((uintptr_t)p.A & 15) == 0;
  scan_step_kernel<T><<<dim3((p.H + per - 1) / per, p.B), kThreads, 0, st>>>(p, state, (T*)y, slots, S, lpc, vec);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_selective_scan(const ScanArgs& p, void* y, float* state_out, float* ckpt, int dtype,
                                  cudaStream_t st) {
  switch (dtype) {
    case 0: return fwd<float>(p, y, state_out, ckpt, st);
    case 1: return fwd<__half>(p, y, state_out, ckpt, st);
    case 2: return fwd<__nv_bfloat16>(p, y, state_out, ckpt, st);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_selective_scan_step(const ScanArgs& p, float* state, void* y, const int* slots, int S, int dtype,
                                       cudaStream_t st) {
  switch (dtype) {
    case 0: return step<float>(p, state, y, slots, S, st);
    case 1: return step<__half>(p, state, y, slots, S, st);
    case 2: return step<__nv_bfloat16>(p, state, y, slots, S, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fc
