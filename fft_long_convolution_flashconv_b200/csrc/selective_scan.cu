// Selective scan: the diagonal SSM whose step size, input and output vectors
// depend on the input, for prompts and for single tokens.
//
//   dt = softplus(delta + dt_bias),  a_n = exp(dt A_n)
//   x_n <- a_n x_n + dt B_n u,  y = (sum_n C_n x_n + D u) silu(z)
//
// A lane holds sixteen steps of one channel in registers and runs through the
// states: it forms a_n and dt B_n u for its steps, runs the recurrence from
// zero, joins the four lanes of a channel by a scan of (product of a, end
// state) over shuffles, runs the recurrence again from the state that enters it
// and adds C_n x_n to its outputs.  The product of a over a lane is
// exp(A_n sum dt), one exponential.  Four lanes of sixteen steps are a 64-step
// block; a warp takes eight channels.  (Eight steps a lane and four channels a warp
// where that leaves too few warps.)
//
// The floor is the special function unit: an exponential a channel, state and step,
// eight cycles a warp.  Measured: 15.4 cycles (9.5 instructions) with sixteen steps
// a lane and every SM full, 18.2 (12.1) with eight; 8 x 768 channels of 1024 steps
// and 16 states in fp16 71 us, one row of 2560 channels of 65536 steps 1.94 ms.
#include "kernels.cuh"
#include "scan.cuh"

namespace fc {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStates = 16;  // states whose B and C are in shared memory at a time
constexpr int TB = kCkptSteps;
constexpr int kMinBlocks = 4;  // resident on an SM
// A lane's steps, and what follows: the lanes of a channel, the channels of a warp and of a block.
template <int TPL_>
struct Shape {
  static constexpr int TPL = TPL_, PAIRS = TPL / 2, VPL = TPL / kVec, TL = TB / TPL, CL = 32 / TL, CH = kWarps * CL;
  // States in flight in a lane, groups of them in one schedule, in the 128 registers that four blocks an SM leave.
  // 2368 channels of 2048 steps, 16 states, fp16: eight steps a lane, batch 4, four states 172 us, two 177; sixteen
  // steps, batch 8, one state 291 us, two states at three blocks of 168 registers 352.
  static constexpr int SG = TPL == 8 ? 4 : 1, kUnroll = TPL == 8 ? 1 : 4;
};

// Place of step t of a block in a row of the B / C tiles: the first four steps
// of every lane, then the next four and so on, so that the 16-byte reads of a
// warp's lanes are contiguous.
template <int TPL>
__device__ __forceinline__ int tile_at(int t) {
  return (t % TPL / 4) * (TB / TPL * 4) + t / TPL * 4 + t % 4;
}

// B and C of up to kStates states of a block: raw vectors into the thread's
// slots, then as floats into the tile that the block computes from.
template <typename T, int TPL>
struct Tiles {
  static constexpr int kRow = TB / 8, kPer = kStates * kRow / kThreads;  // vectors of a row, of a thread (B, and C)
  const T *Bt, *Ct;
  T* slot;  // 2 kPer * 8 elements
  __device__ __forceinline__ void fetch(const ScanArgs& p, int s0, int ns, int tb, int n) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x + j * kThreads, s = i / kRow, t0 = tb + i % kRow * 8;
      if (s < ns) {
        fetch8(slot + j * 8, Bt + (s0 + s) * p.Bt.rs, t0, p.L, n, p.Bt.vec);
        fetch8(slot + (kPer + j) * 8, Ct + (s0 + s) * p.Ct.rs, t0, p.L, n, p.Ct.vec);
      }
    }
  }
  // The same of rows on two-byte boundaries, where the block lies inside the sequence: all loads before the first
  // is used (threads without a row of their own repeat the last).
  __device__ __forceinline__ void fetch_odd(const ScanArgs& p, int s0, int ns, int tb) const {
    Wide<T> b[kPer], c[kPer];
    long long at[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x + j * kThreads;
      at[j] = s0 + min(i / kRow, ns - 1);
      b[j].load(Bt + at[j] * p.Bt.rs + tb + i % kRow * 8);
      c[j].load(Ct + at[j] * p.Ct.rs + tb + i % kRow * 8);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = threadIdx.x + j * kThreads;
      b[j].put(slot + j * 8, Bt + at[j] * p.Bt.rs + tb + i % kRow * 8);
      c[j].put(slot + (kPer + j) * 8, Ct + at[j] * p.Ct.rs + tb + i % kRow * 8);
    }
  }
  // Rows from ns on, which fill up a group of states, are zeros.
  __device__ __forceinline__ void store(float* buf, int ns, int tb, int n) const {
#pragma unroll
    for (int j = 0; j < 2 * kPer; ++j) {
      const int i = threadIdx.x + j % kPer * kThreads, s = i / kRow, k = i % kRow;
      float v[8] = {};
      if (s < ns) take8(slot + j * 8, tb + k * 8, n, v);
      float* d = buf + (j / kPer * kStates + s) * TB;
      *reinterpret_cast<float4*>(d + tile_at<TPL>(k * 8)) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(d + tile_at<TPL>(k * 8 + 4)) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
};

// Step D of the scan over a channel's lanes: lane t joins what lane t - D
// holds, h = P h' + h and P = P P' (not after the last step); lanes below D keep
// theirs.  One predicated instruction each instead of a branch keeps several
// states' work in one schedule.
template <int TL, int D>
__device__ __forceinline__ void join(float& h, float& P) {
  constexpr int kClamp = (32 - TL) << 8;
  if (D * 2 < TL)
    asm volatile(
        "{ .reg .pred q; .reg .f32 t, s; shfl.sync.up.b32 t|q, %0, %2, %3, -1; shfl.sync.up.b32 s, %1, %2, %3, -1;\n"
        "@q fma.rn.f32 %0, %1, t, %0; @q mul.rn.f32 %1, %1, s; }"
        : "+f"(h), "+f"(P)
        : "n"(D), "n"(kClamp));
  else
    asm volatile("{ .reg .pred q; .reg .f32 t; shfl.sync.up.b32 t|q, %0, %2, %3, -1; @q fma.rn.f32 %0, %1, t, %0; }"
                 : "+f"(h)
                 : "f"(P), "n"(D), "n"(kClamp));
}
// h of the lane before; the first lane of a channel keeps `first`.
template <int TL>
__device__ __forceinline__ float before(float h, float first) {
  asm volatile("{ .reg .pred q; .reg .f32 t; shfl.sync.up.b32 t|q, %1, 1, %2, -1; @q mov.f32 %0, t; }"
               : "+f"(first)
               : "f"(h), "n"((32 - TL) << 8));
  return first;
}

// The steps of a lane: step sizes, dt u and the outputs so far.
template <int PAIRS>
struct Lane {
  float2 dt[PAIRS], du[PAIRS], o[PAIRS];
  float sum;  // of dt
};

// SG states of a block, rows from Bs on, for a lane's steps: o += C x.  As: the
// states' A log2(e), rows of CH channels; x0s: the state entering the first lane
// of a channel, zeros for the others; x1s: where the last lane's end state goes
// (the others write to a place that nothing reads).
template <typename S, bool CKPT>
__device__ __forceinline__ void run_states(const float* Bs, const float* As, const float* x0s, uint32_t x1s, int tl,
                                           Lane<S::PAIRS>& l, bool keep, float* ckpt, int nlive) {
  constexpr int SG = S::SG, PAIRS = S::PAIRS, TPL = S::TPL, TL = S::TL, CH = S::CH;
  float2 a[SG][PAIRS], w[SG][PAIRS];
  float h[SG], P[SG], x0[SG];
#pragma unroll
  for (int q = 0; q < SG; ++q) {
    const float4* Bp = reinterpret_cast<const float4*>(Bs + q * TB) + tl;
    const float A2 = As[q * CH];
    x0[q] = x0s[q * CH];
#pragma unroll
    for (int i = 0; i < TPL / 4; ++i) {
      const float4 v = Bp[i * TL];
      w[q][2 * i] = mul2(l.du[2 * i], make_float2(v.x, v.y));
      w[q][2 * i + 1] = mul2(l.du[2 * i + 1], make_float2(v.z, v.w));
    }
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const float2 e = mul2(l.dt[i], both(A2));
      a[q][i] = make_float2(ex2(e.x), ex2(e.y));
    }
    P[q] = ex2(l.sum * A2);
  }
#pragma unroll
  for (int q = 0; q < SG; ++q) {
    float v = fmaf(a[q][0].y, w[q][0].x, w[q][0].y);
#pragma unroll
    for (int i = 1; i < PAIRS; ++i) {
      v = fmaf(a[q][i].x, v, w[q][i].x);
      v = fmaf(a[q][i].y, v, w[q][i].y);
    }
    h[q] = fmaf(P[q], x0[q], v);
  }
  // states at the end of every lane
#pragma unroll
  for (int q = 0; q < SG; ++q) join<TL, 1>(h[q], P[q]);
#pragma unroll
  for (int q = 0; q < SG; ++q) join<TL, 2>(h[q], P[q]);
  if constexpr (TL > 4) {
#pragma unroll
    for (int q = 0; q < SG; ++q) join<TL, 4>(h[q], P[q]);
  }
#pragma unroll
  for (int q = 0; q < SG; ++q) {
    put_shared(x1s + q * CH * 4, h[q]);
    const float4* Cp = reinterpret_cast<const float4*>(Bs + (kStates + q) * TB) + tl;
    float v = before<TL>(h[q], x0[q]);
    if (CKPT) put_global(keep && q < nlive, ckpt + q, v);
#pragma unroll
    for (int i = 0; i < TPL / 4; ++i) {
      const float4 cv = Cp[i * TL];
      float2 x, z;
      x.x = v = fmaf(a[q][2 * i].x, v, w[q][2 * i].x);
      x.y = v = fmaf(a[q][2 * i].y, v, w[q][2 * i].y);
      z.x = v = fmaf(a[q][2 * i + 1].x, v, w[q][2 * i + 1].x);
      z.y = v = fmaf(a[q][2 * i + 1].y, v, w[q][2 * i + 1].y);
      l.o[2 * i] = fma2(make_float2(cv.x, cv.y), x, l.o[2 * i]);
      l.o[2 * i + 1] = fma2(make_float2(cv.z, cv.w), z, l.o[2 * i + 1]);
    }
  }
}

// Shared memory of a scan block, in floats from the start.
template <typename T, int TPL>
struct Layout {
  using S = Shape<TPL>;
  static constexpr int VPL = S::VPL, CH = S::CH;
  static constexpr int bc = 0;                  // [2][2 kStates][TB] B and C
  static constexpr int raw = 4 * kStates * TB;  // [2 kPer][8] T of a thread: B and C on their way
  static constexpr int in = raw + 2 * Tiles<T, TPL>::kPer * 8 * kThreads * (int)sizeof(T) / 4;  // [5][VPL] T vectors
  static constexpr int states = in + 5 * VPL * 8 * kThreads * (int)sizeof(T) / 4;
  // [4][Np][CH]: A log2(e); entering states; zeros; what nothing reads
  static size_t bytes(int Np) { return (size_t)(states + 4 * Np * CH) * 4; }
};

// A block of four warps takes CH channels of a group.
// ODD: 16-bit rows, none of them on 16-byte boundaries (an odd L, mostly).
template <typename T, int TPL, bool CKPT, bool ODD>
__global__ __launch_bounds__(kThreads, kMinBlocks) void scan_kernel(ScanArgs p, Segments sg, T* y,
                                                                                float* state_out, float* ckpt,
                                                                                int tiles) {
  using S = Shape<TPL>;
  using Sm = Layout<T, TPL>;
  constexpr int TL = S::TL, CL = S::CL, CH = S::CH, VPL = S::VPL, SG = S::SG;
  static_assert(kStates % SG == 0, "states come in whole groups");
  extern __shared__ float4 smem4[];
  float* const sm = reinterpret_cast<float*>(smem4);
  const int N = p.N, chunks = (N + kStates - 1) / kStates, Np = chunks * kStates;
  float* const bc = sm + Sm::bc;
  float* const As = sm + Sm::states;
  float* const xs = As + Np * CH;
  const int tid = threadIdx.x, lane = tid & 31, tl = lane % TL, c = (tid >> 5) * CL + lane / TL;
  const int E = p.H / p.G, nseg = sg.count;
  const int seg = blockIdx.x % nseg, tile = blockIdx.x / nseg % tiles, bg = blockIdx.x / nseg / tiles;
  const int b = bg / p.G, g = bg % p.G;
  const int n = row_length(p.lengths, b, p.L);
  for (int i = tid; i < Np * CH; i += kThreads) {
    const int s = i / CH, cc = i % CH, hh = g * E + tile * CH + cc;
    const bool ok = tile * CH + cc < E && s < N;
    const long long row = (long long)b * p.H + hh;
    As[i] = ok ? __ldg(p.A + (long long)hh * N + s) * kLog2e : 0.f;
    xs[i] = !ok          ? 0.f
            : sg.state   ? __ldg(sg.state + (row * nseg + seg) * N + s)
            : p.state_in ? __ldg(p.state_in + row * N + s)
                         : 0.f;
    xs[Np * CH + i] = 0.f;
  }
  const float* const x0s = (tl == 0 ? xs : xs + Np * CH) + c;
  const uint32_t x1s = shared_addr((tl == TL - 1 ? xs : xs + 2 * Np * CH) + c);
  const bool live = tile * CH + c < E;
  const int h = g * E + (live ? tile * CH + c : 0);
  const float Dh = p.D ? __ldg(p.D + h) : 0.f, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
  const T* u = (const T*)p.u.p + b * p.u.bs + h * p.u.rs;
  const T* delta = (const T*)p.delta.p + b * p.delta.bs + h * p.delta.rs;
  const T* z = p.z.p ? (const T*)p.z.p + b * p.z.bs + h * p.z.rs : nullptr;
  T* yr = y + ((long long)b * p.H + h) * p.L;
  const Tiles<T, TPL> next{(const T*)p.Bt.p + b * p.Bt.bs + g * p.Bt.gs, (const T*)p.Ct.p + b * p.Ct.bs + g * p.Ct.gs,
                      reinterpret_cast<T*>(sm + Sm::raw) + tid * 2 * Tiles<T, TPL>::kPer * 8};
  T* const in = reinterpret_cast<T*>(sm + Sm::in) + tid * 8;
  const int nck = (p.L + TB - 1) / TB;
  const int first = seg * sg.blocks, last = min(nck, first + sg.blocks), end = min(last, (n + TB - 1) / TB);

  Lane<S::PAIRS> l;
  // u and delta of even and odd blocks, z
  auto slot = [&](int which, int j) { return in + (which * VPL + j) * kThreads * 8; };
  auto fetch = [&](int k) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int t0 = k * TB + tl * TPL + j * 8;
      fetch8(slot((k & 1) * 2, j), u, t0, p.L, n, p.u.vec);
      fetch8(slot((k & 1) * 2 + 1, j), delta, t0, p.L, n, p.delta.vec);
    }
  };
  // step sizes of block k: dt = 0 behind the row's end keeps the state
  auto steps = [&](int k) {
    l.sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int t0 = k * TB + tl * TPL + j * 8;
      float uv[8], dv[8];
      take8(slot((k & 1) * 2, j), t0, n, uv);
      take8(slot((k & 1) * 2 + 1, j), t0, INT_MAX, dv);
      float2* d = l.dt + 4 * j;
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = add2(make_float2(dv[2 * i], dv[2 * i + 1]), both(bias));
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = softplus2(d[i]);
      }
      if (t0 + 8 > n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (t0 + 2 * i >= n) d[i].x = 0.f;
          if (t0 + 2 * i + 1 >= n) d[i].y = 0.f;
        }
      }
      float2 sum = add2(add2(d[0], d[1]), add2(d[2], d[3]));
      l.sum += sum.x + sum.y;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        l.du[4 * j + i] = mul2(d[i], make_float2(uv[2 * i], uv[2 * i + 1]));
        l.o[4 * j + i] = mul2(both(Dh), make_float2(uv[2 * i], uv[2 * i + 1]));
      }
    }
  };

  if (first < end) {
    next.fetch(p, 0, min(N, kStates), first * TB, n);
    fetch(first);
    fetched();
    next.store(bc, min(N, kStates), first * TB, n);
  }
  __syncthreads();
  int it = 0;
  for (int k = first; k < end; ++k) {
    steps(k);
    // Rows on two-byte boundaries inside the sequence: this block's gate, the next one's u and delta and the next B
    // and C tile, loaded together.
    const bool together = ODD && k > 0 && k + 1 < end && (k + 2) * TB + 8 <= p.L;
    if (together) {
      if constexpr (ODD) {
        const T* zz = z ? z : u;
        Wide<T> q[3][VPL];
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int t0 = k * TB + tl * TPL + j * 8;
          q[0][j].load(u + t0 + TB);
          q[1][j].load(delta + t0 + TB);
          q[2][j].load(zz + t0);
        }
        next.fetch_odd(p, chunks > 1 ? kStates : 0, min(N - (chunks > 1 ? kStates : 0), kStates),
                       (chunks > 1 ? k : k + 1) * TB);
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const int t0 = k * TB + tl * TPL + j * 8;
          q[0][j].put(slot(((k + 1) & 1) * 2, j), u + t0 + TB);
          q[1][j].put(slot(((k + 1) & 1) * 2 + 1, j), delta + t0 + TB);
          q[2][j].put(slot(4, j), zz + t0);
        }
      }
    } else {
      if (z) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) fetch8(slot(4, j), z, k * TB + tl * TPL + j * 8, p.L, n, p.z.vec);
      }
      if (k + 1 < end) fetch(k + 1);
    }
    float* ck = CKPT ? ckpt + (((long long)b * p.H + h) * nck + k) * N : nullptr;
    for (int ch = 0; ch < chunks; ++ch, ++it) {
      const int s0 = ch * kStates, ns = min(N - s0, kStates);
      const bool more = ch + 1 < chunks || k + 1 < end;
      const int sn = ch + 1 < chunks ? s0 + kStates : 0, tbn = (ch + 1 < chunks ? k : k + 1) * TB;
      if (more && !(together && ch == 0)) {
        if (ODD && k > 0 && (k + 2) * TB + 8 <= p.L) {
          if constexpr (ODD) next.fetch_odd(p, sn, min(N - sn, kStates), tbn);
        } else {
          next.fetch(p, sn, min(N - sn, kStates), tbn, n);
        }
      }
      const float* Bs = bc + (it & 1) * 2 * kStates * TB;
#pragma unroll S::kUnroll
      for (int e = 0; e < ns; e += SG)
        run_states<S, CKPT>(Bs + e * TB, As + (s0 + e) * CH + c, x0s + (s0 + e) * CH, x1s + (s0 + e) * CH * 4, tl,
                                  l, live && tl == 0, ck + s0 + e, ns - e);
      fetched();
      if (more) next.store(bc + ((it + 1) & 1) * 2 * kStates * TB, min(N - sn, kStates), tbn, n);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int t0 = k * TB + tl * TPL + j * 8;
      float v[8], w[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = l.o[4 * j + i].x;
        v[2 * i + 1] = l.o[4 * j + i].y;
      }
      if (z) {
        take8(slot(4, j), t0, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= silu(w[i]);
      }
      if (live && t0 < p.L) store8(yr, t0, p.L, n, p.out_vec, v);
    }
  }
  for (int k = max(first, end); k < last; ++k) {  // behind the row's end
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int t0 = k * TB + tl * TPL + j * 8;
      float v[8] = {};
      if (live && t0 < p.L) store8(yr, t0, p.L, n, p.out_vec, v);
    }
  }
  if (state_out && seg == nseg - 1) {
    for (int i = tid; i < N * CH; i += kThreads) {
      const int cc = i / N, s = i % N;
      if (tile * CH + cc < E) state_out[((long long)b * p.H + g * E + tile * CH + cc) * N + s] = xs[s * CH + cc];
    }
  }
}

// One token.  LPC lanes share a channel, four states (one 16-byte access where N
// is a multiple of four) of each; a thread takes kTok channels, whose states it
// loads before anything is known of the slot but its range, and B and C once for
// all.  Lane j % LPC of a channel's lanes computes the step size and the gate of
// its j-th channel for the others.
constexpr int kTok = 4;

template <typename T, bool VEC, int LPC>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(ScanArgs p, float* state, T* y, const int* slots, int S) {
  constexpr int per = kThreads / LPC, own = (kTok + LPC - 1) / LPC;  // channels apart; those a lane answers for
  const int b = blockIdx.y, sub = threadIdx.x % LPC, N = p.N;
  const int h0 = blockIdx.x * per * kTok + threadIdx.x / LPC;  // channels h0, h0 + per, ...
  const int raw = slots ? __ldg(slots + b) : b;
  float* const pool = state + (raw >= 0 && raw < S ? (long long)raw * p.H * N : 0);
  const int s = sub * 4;
  float4 x[kTok], A[kTok];
  auto load4 = [&](const float* q, int at) {
    if (VEC) return at < N ? *reinterpret_cast<const float4*>(q + at) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(at < N ? q[at] : 0.f, at + 1 < N ? q[at + 1] : 0.f, at + 2 < N ? q[at + 2] : 0.f,
                       at + 3 < N ? q[at + 3] : 0.f);
  };
#pragma unroll
  for (int j = 0; j < kTok; ++j) {  // channels behind the last read the last one's
    const long long at = (long long)min(h0 + j * per, p.H - 1) * N;
    x[j] = load4(pool + at, s);
    A[j] = load4(p.A + at, s);
  }
  // step size, u and gate of the channels that this lane answers for: j = e LPC + sub
  float dt[own], u[own], z[own];
#pragma unroll
  for (int e = 0; e < own; ++e) {
    const int h = min(h0 + (e * LPC + sub) % kTok * per, p.H - 1);
    u[e] = IO<T>::ldplain((const T*)p.u.p + b * p.u.bs + h * p.u.rs);
    dt[e] = IO<T>::ldplain((const T*)p.delta.p + b * p.delta.bs + h * p.delta.rs);
    if (p.dt_bias) dt[e] += __ldg(p.dt_bias + h);
    z[e] = p.z.p ? IO<T>::ldplain((const T*)p.z.p + b * p.z.bs + h * p.z.rs) : 0.f;
  }
  float Bv[4], Cv[4];
  int group = -1;
  const int slot = batch_slot(slots, b, S);
#pragma unroll
  for (int e = 0; e < own; ++e) {
    if (p.softplus) dt[e] = softplus(dt[e]);
    z[e] = p.z.p ? silu(z[e]) : 1.f;
  }
#pragma unroll
  for (int j = 0; j < kTok; ++j) {
    const int h = h0 + j * per;
    const float d = __shfl_sync(~0u, dt[j / LPC], j % LPC, LPC), uj = __shfl_sync(~0u, u[j / LPC], j % LPC, LPC);
    const float du = d * uj, d2 = d * kLog2e;
    const int g = p.G == 1 ? 0 : min(h, p.H - 1) / (p.H / p.G);
    const T* Bt = (const T*)p.Bt.p + b * p.Bt.bs + g * p.Bt.gs;
    const T* Ct = (const T*)p.Ct.p + b * p.Ct.bs + g * p.Ct.gs;
    if (g != group) {  // the lane's first four states
      group = g;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Bv[i] = s + i < N ? IO<T>::ldplain(Bt + (s + i) * p.Bt.rs) : 0.f;
        Cv[i] = s + i < N ? IO<T>::ldplain(Ct + (s + i) * p.Ct.rs) : 0.f;
      }
    }
    const bool on = h < p.H && slot >= 0;
    float* const xp = pool + (long long)h * N;
    float acc = 0.f;
    auto update = [&](int q, float4 xv, float4 av, const float (&bv)[4], const float (&cv)[4]) {
      xv = make_float4(fmaf(ex2(d2 * av.x), xv.x, du * bv[0]), fmaf(ex2(d2 * av.y), xv.y, du * bv[1]),
                       fmaf(ex2(d2 * av.z), xv.z, du * bv[2]), fmaf(ex2(d2 * av.w), xv.w, du * bv[3]));
      acc = fmaf(cv[0], xv.x, fmaf(cv[1], xv.y, fmaf(cv[2], xv.z, fmaf(cv[3], xv.w, acc))));
      if (!on || q >= N) return;
      if (VEC) {
        *reinterpret_cast<float4*>(xp + q) = xv;
      } else {
        xp[q] = xv.x;
        if (q + 1 < N) xp[q + 1] = xv.y;
        if (q + 2 < N) xp[q + 2] = xv.z;
        if (q + 3 < N) xp[q + 3] = xv.w;
      }
    };
    update(s, x[j], A[j], Bv, Cv);
    if (LPC == 32 && on) {  // more than 128 states
      for (int q = s + 4 * LPC; q < N; q += 4 * LPC) {
        float bv[4], cv[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          bv[i] = q + i < N ? IO<T>::ldplain(Bt + (q + i) * p.Bt.rs) : 0.f;
          cv[i] = q + i < N ? IO<T>::ldplain(Ct + (q + i) * p.Ct.rs) : 0.f;
        }
        update(q, load4(xp, q), load4(p.A + (long long)h * N, q), bv, cv);
      }
    }
#pragma unroll
    for (int e = LPC / 2; e; e >>= 1) acc += __shfl_xor_sync(~0u, acc, e);
    if (h < p.H && sub == j % LPC) {
      const float o = fmaf(p.D ? __ldg(p.D + h) : 0.f, uj, acc) * z[j / LPC];
      IO<T>::st(y + (long long)b * p.H + h, slot < 0 ? 0.f : o);
    }
  }
}

template <typename T, int TPL, bool CKPT, bool ODD>
cudaError_t run(const ScanArgs& p, const Segments& sg, void* y, float* state_out, float* ckpt, cudaStream_t st) {
  constexpr int CH = Shape<TPL>::CH;
  const int tiles = (p.H / p.G + CH - 1) / CH;
  const size_t smem = Layout<T, TPL>::bytes((p.N + kStates - 1) / kStates * kStates);
  const cudaError_t e = smem_optin<scan_kernel<T, TPL, CKPT, ODD>>(smem);
  if (e != cudaSuccess) return e;
  scan_kernel<T, TPL, CKPT, ODD><<<(unsigned)((long long)tiles * p.B * p.G * sg.count), kThreads, smem, st>>>(
      p, sg, (T*)y, state_out, ckpt, tiles);
  return cudaGetLastError();
}
template <typename T, int TPL>
cudaError_t run(const ScanArgs& p, const Segments& sg, void* y, float* state_out, float* ckpt, cudaStream_t st) {
  if constexpr (sizeof(T) == 2) {
    // a kernel of its own (8 x 768 x 2047, fp16: 200 -> 171 us; the branch in the other one cost 3 to 4%)
    if (!p.u.vec && !p.delta.vec && !(p.z.p && p.z.vec) && !p.Bt.vec && !p.Ct.vec)
      return ckpt ? run<T, TPL, true, true>(p, sg, y, state_out, ckpt, st)
                  : run<T, TPL, false, true>(p, sg, y, state_out, nullptr, st);
  }
  return ckpt ? run<T, TPL, true, false>(p, sg, y, state_out, ckpt, st)
              : run<T, TPL, false, false>(p, sg, y, state_out, nullptr, st);
}

template <typename T>
cudaError_t fwd(const ScanArgs& p, int tpl, const Segments& sg, void* y, float* state_out, float* ckpt,
                cudaStream_t st) {
  return tpl == 8 ? run<T, 8>(p, sg, y, state_out, ckpt, st) : run<T, 16>(p, sg, y, state_out, ckpt, st);
}

struct Plan {
  int tpl;
  Segments sg;
};

// Steps of a lane and segments of a row.  Sixteen steps need the fewest
// instructions (four thread blocks an SM: 15.4 cycles a warp, state and step,
// eight: 18.2) but leave half as many warps.  Segments fill the SMs where
// channels are few, for a first pass over the segments' end states: 128 channels of
// 8192 steps took 373 us in one piece.  The cheapest of the choices is taken.
Plan plan(int B, int H, int L, int N, int G) {
  const int all = (L + TB - 1) / TB, sms = num_sms();
  Plan best{16, {1, all, nullptr, nullptr}};
  float least = -1.f;
  for (int tpl = 8; tpl <= 16; tpl += 8) {
    const int ch = kWarps * 32 / (TB / tpl);
    const float c = tpl == 8 ? 45.f : 95.f, d = tpl == 8 ? 31.5f : 49.f;
    const long long ctas = (long long)B * G * ((H / G + ch - 1) / ch);
    for (int want = 1; want <= 64 && (want == 1 || ctas * (want - 1) < 16 * sms); ++want) {
      const int blocks = (all + want - 1) / want, count = (all + blocks - 1) / blocks;
      if (count != want || (count > 1 && blocks < 4)) continue;
      const float t = scan_cost(ctas * count, blocks, kMinBlocks, c, d, sms) +
                      (count > 1 ? ends_cost(B, H, G, N, count, blocks, sms) : 0.f);
      if (least < 0.f || t < least) {
        least = t;
        best = {tpl, {count, blocks, nullptr, nullptr}};
      }
    }
  }
  return best;
}

template <typename T, bool VEC>
cudaError_t step_v(const ScanArgs& p, float* state, void* y, const int* slots, int S, cudaStream_t st) {
  int lpc = 1;
  while (lpc < 32 && lpc * 4 < p.N) lpc *= 2;
  const int per = kThreads / lpc * kTok;
  const dim3 grid((p.H + per - 1) / per, p.B);
  switch (lpc) {
    case 1: scan_step_kernel<T, VEC, 1><<<grid, kThreads, 0, st>>>(p, state, (T*)y, slots, S); break;
    case 2: scan_step_kernel<T, VEC, 2><<<grid, kThreads, 0, st>>>(p, state, (T*)y, slots, S); break;
    case 4: scan_step_kernel<T, VEC, 4><<<grid, kThreads, 0, st>>>(p, state, (T*)y, slots, S); break;
    case 8: scan_step_kernel<T, VEC, 8><<<grid, kThreads, 0, st>>>(p, state, (T*)y, slots, S); break;
    case 16: scan_step_kernel<T, VEC, 16><<<grid, kThreads, 0, st>>>(p, state, (T*)y, slots, S); break;
    default: scan_step_kernel<T, VEC, 32><<<grid, kThreads, 0, st>>>(p, state, (T*)y, slots, S); break;
  }
  return cudaGetLastError();
}
template <typename T>
cudaError_t step(const ScanArgs& p, float* state, void* y, const int* slots, int S, cudaStream_t st) {
  const bool vec = p.N % 4 == 0 && ((uintptr_t)state & 15) == 0 && ((uintptr_t)p.A & 15) == 0;
  return vec ? step_v<T, true>(p, state, y, slots, S, st) : step_v<T, false>(p, state, y, slots, S, st);
}

}  // namespace

int selective_scan_lane_steps(int B, int H, int L, int N, int G) { return plan(B, H, L, N, G).tpl; }

size_t selective_scan_workspace_bytes(int B, int H, int L, int N, int G) {
  return segments_bytes(plan(B, H, L, N, G).sg, B, H, N);
}

cudaError_t launch_selective_scan(const ScanArgs& p, void* y, float* state_out, float* ckpt, void* workspace, int dtype,
                                  cudaStream_t st) {
  Plan pl = plan(p.B, p.H, p.L, p.N, p.G);
  place_segments(&pl.sg, workspace, p.B, p.H, p.N);
  if (pl.sg.count > 1) {
    const cudaError_t e = launch_segment_states(p, pl.sg, p.state_in, false, dtype, st);
    if (e != cudaSuccess) return e;
  }
  switch (dtype) {
    case 0: return fwd<float>(p, pl.tpl, pl.sg, y, state_out, ckpt, st);
    case 1: return fwd<__half>(p, pl.tpl, pl.sg, y, state_out, ckpt, st);
    case 2: return fwd<__nv_bfloat16>(p, pl.tpl, pl.sg, y, state_out, ckpt, st);
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
