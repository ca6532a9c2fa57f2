// Backward pass of the selective scan.
//
// With dyp = dy silu(z) and the adjoint g_n[t] = C_n[t] dyp[t] + a_n[t+1] g_n[t+1]
// of the state x_n[t]:
//   du = D dyp + dt sum_n g_n B_n
//   ddt = u sum_n g_n B_n + sum_n A_n g_n a_n x_n[t-1],  ddelta = ddt softplus'
//   dA_n = sum_{b,t} dt g_n a_n x_n[t-1],  dD = sum dyp u,  ddt_bias = sum ddelta
//   dB_n[t] = sum_h g_n dt u,  dC_n[t] = sum_h dyp x_n,  dz = dy y silu'(z)
//
// Measured: 35 instructions and 56 cycles a warp, state and step, bound by their
// issue and latency (62% of its slots with 14 warps an SM); 217 us for 4 x 1024 channels of 2048 steps, 16 states,
// bf16.
//
// A lane holds eight steps of one channel; eight lanes are a channel's 64-step
// block, a warp takes four channels and walks through the blocks from the last
// to the first.  In a block it runs each state forward again from the kept state
// that enters the block, then its adjoint backward; both recurrences are joined
// over a channel's lanes by shuffles, as in the forward kernel.
//
// dB and dC are sums over the group's channels: shuffles add the four lanes that
// hold the same steps (each keeps a quarter of them), the block's warps are added
// in shared memory and the blocks by scan_sum_bc_kernel, always in the same order,
// so results do not change from run to run.  (Adding up the lanes by products with
// ones on the tensor cores cost more instructions, most of them moves into operand
// registers; two channels a lane would halve the shuffles but spill at the 168
// registers that three blocks an SM leave, and gain nothing with two: 1556 to
// 1799 us for a training step of 4 x 1024 channels of 8192 steps, when this form
// took 1537.)
#include "kernels.cuh"
#include "scan.cuh"

namespace fc {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStates = 8;  // states whose tiles are in shared memory at a time
constexpr int kLaneStates = 16;  // up to so many states a lane keeps its own dA (8 KB: four blocks an SM still fit)
constexpr int kMinBlocks = 4;  // resident on an SM: 128 registers a thread
constexpr int TPL = 8, TL = 8, CL = 4, TB = kCkptSteps, CH = kWarps * CL, PAIRS = TPL / 2;
static_assert(TB == TL * TPL, "a block of steps is what a channel's lanes hold");

struct BwdOut {
  void *du, *ddelta, *dz;
  const float* ckpt;
  const float* dstate_out;
  float* dstate_in;
  float* part_bc;  // [tiles][2][B][G][N][L]
  float* part_a;   // [B][segments][H][N]
  float* part_d;   // [2][B][segments][H]: dD, ddt_bias
};

// Step D of the scan over a channel's lanes, which are four lanes apart: from the
// lanes before (UP) or behind.
template <bool UP, int D>
__device__ __forceinline__ void join(float& h, float& P) {
  if constexpr (D * 2 == TL) {  // the product is not needed after the last step
    if constexpr (UP)
      asm volatile("{ .reg .pred q; .reg .f32 t; shfl.sync.up.b32 t|q, %0, %2, 0, -1; @q fma.rn.f32 %0, %1, t, %0; }"
                   : "+f"(h)
                   : "f"(P), "n"(D * CL));
    else
      asm volatile("{ .reg .pred q; .reg .f32 t; shfl.sync.down.b32 t|q, %0, %2, 31, -1; @q fma.rn.f32 %0, %1, t, %0; }"
                   : "+f"(h)
                   : "f"(P), "n"(D * CL));
  } else if constexpr (UP) {
    asm volatile(
        "{ .reg .pred q; .reg .f32 t, s; shfl.sync.up.b32 t|q, %0, %2, 0, -1; shfl.sync.up.b32 s, %1, %2, 0, -1;\n"
        "@q fma.rn.f32 %0, %1, t, %0; @q mul.rn.f32 %1, %1, s; }"
        : "+f"(h), "+f"(P)
        : "n"(D * CL));
  } else {
    asm volatile(
        "{ .reg .pred q; .reg .f32 t, s; shfl.sync.down.b32 t|q, %0, %2, 31, -1; shfl.sync.down.b32 s, %1, %2, 31, -1;\n"
        "@q fma.rn.f32 %0, %1, t, %0; @q mul.rn.f32 %1, %1, s; }"
        : "+f"(h), "+f"(P)
        : "n"(D * CL));
  }
}
// The neighbour's h; the first (last) lane of a channel keeps `edge`.
template <bool UP>
__device__ __forceinline__ float neighbour(float h, float edge) {
  if constexpr (UP)
    asm volatile("{ .reg .pred q; .reg .f32 t; shfl.sync.up.b32 t|q, %1, %2, 0, -1; @q mov.f32 %0, t; }"
                 : "+f"(edge)
                 : "f"(h), "n"(CL));
  else
    asm volatile("{ .reg .pred q; .reg .f32 t; shfl.sync.down.b32 t|q, %1, %2, 31, -1; @q mov.f32 %0, t; }"
                 : "+f"(edge)
                 : "f"(h), "n"(CL));
  return edge;
}

// Sum v (eight steps) over the four lanes that hold the same steps, lane ^ 1 and
// lane ^ 2: lane 4 tl + cl returns the sums of elements 2 cl and 2 cl + 1.
__device__ __forceinline__ float2 sum_channels(const float2 (&v)[PAIRS], int cl) {
  const bool hi = cl & 2, odd = cl & 1;
  float2 w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 give = hi ? v[i] : v[i + 2], keep = hi ? v[i + 2] : v[i];
    w[i] = add2(keep, make_float2(__shfl_xor_sync(~0u, give.x, 2), __shfl_xor_sync(~0u, give.y, 2)));
  }
  const float2 give = odd ? w[0] : w[1], keep = odd ? w[1] : w[0];
  return add2(keep, make_float2(__shfl_xor_sync(~0u, give.x, 1), __shfl_xor_sync(~0u, give.y, 1)));
}

// Place of step t in a row of the B / C tiles: the first four steps of every
// lane, then the others, so that the 16-byte reads of a warp's lanes are contiguous.
__device__ __forceinline__ int tile_at(int t) { return (t & 4) * TL + (t >> 3) * 4 + (t & 3); }

template <typename T>
struct Sm {
  T in[2][4][kThreads][8];                          // u, delta, dy, z of even and odd blocks
  T raw[kStates * TB / 8 * 2 / kThreads][kThreads][8];  // B and C on their way
  float tile[2][2][kStates][TB];                    // B and C as floats
  float sums[kWarps][kStates][2][TB];               // dB, dC of a warp's channels
  float ck[2][kStates][CH];                         // states entering the block
  float zero[kStates][CH];                          // for the lanes that none enters
  // [Np][CH] each: A, entering adjoint, what nothing reads; then dA, of every lane ([Np][kThreads], up to kLaneStates
  // states) or of the channels (twice [Np][CH], the second never read)
};

template <typename T>
__global__ __launch_bounds__(kThreads, kMinBlocks) void scan_bwd_kernel(ScanArgs p, BwdOut q, Segments sg, int tiles) {
  extern __shared__ float4 smem4[];
  Sm<T>& sm = *reinterpret_cast<Sm<T>*>(smem4);
  const int N = p.N, chunks = (N + kStates - 1) / kStates, Np = chunks * kStates;
  float* const As = reinterpret_cast<float*>(&sm + 1);  // [Np][CH]
  float* const gs = As + Np * CH;  // as large, and as much behind it that nothing reads
  float* const das = gs + 2 * Np * CH;
  const bool lanes = Np <= kLaneStates;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tl = lane / CL, cl = lane % CL, c = warp * CL + cl;
  const int E = p.H / p.G;
  const int seg = blockIdx.x % sg.count, tile = blockIdx.x / sg.count % tiles, bg = blockIdx.x / sg.count / tiles;
  const int b = bg / p.G, g = bg % p.G;
  const bool live = tile * CH + c < E;
  const int h = g * E + (live ? tile * CH + c : 0);
  const long long row = (long long)b * p.H + h;
  const int n = row_length(p.lengths, b, p.L);
  for (int i = tid; i < Np * CH; i += kThreads) {
    const int s = i / CH, cc = i % CH, hh = g * E + tile * CH + cc;
    const bool ok = tile * CH + cc < E && s < N;
    const long long r = (long long)b * p.H + hh;
    As[i] = ok ? __ldg(p.A + (long long)hh * N + s) : 0.f;
    gs[i] = !ok            ? 0.f
            : sg.state     ? __ldg(sg.state + (r * sg.count + seg) * N + s)
            : q.dstate_out ? __ldg(q.dstate_out + r * N + s)
                           : 0.f;
    if (i < kStates * CH) sm.zero[0][i] = 0.f;
  }
  for (int i = tid; i < Np * (lanes ? kThreads : 2 * CH); i += kThreads) das[i] = 0.f;
  float* const da_at = das + (lanes ? tid : (tl == 0 ? 0 : Np * CH) + c);
  const int da_step = lanes ? kThreads : CH;
  const uint32_t r1s = shared_addr(tl == 0 ? gs + c : gs + Np * CH + c);
  const T* u = (const T*)p.u.p + b * p.u.bs + h * p.u.rs;
  const T* delta = (const T*)p.delta.p + b * p.delta.bs + h * p.delta.rs;
  const T* dy = (const T*)p.dy.p + b * p.dy.bs + h * p.dy.rs;
  const T* z = p.z.p ? (const T*)p.z.p + b * p.z.bs + h * p.z.rs : nullptr;
  const T* Bt = (const T*)p.Bt.p + b * p.Bt.bs + g * p.Bt.gs;
  const T* Ct = (const T*)p.Ct.p + b * p.Ct.bs + g * p.Ct.gs;
  const float Dh = p.D ? __ldg(p.D + h) : 0.f, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
  const int nck = (p.L + TB - 1) / TB;
  const int first = seg * sg.blocks, last = min(nck, first + sg.blocks), end = min(last, (n + TB - 1) / TB);
  float* pbc = q.part_bc + ((long long)tile * 2 * p.B * p.G + bg) * N * p.L;  // dB; dC is B G N L further
  const long long pstep = (long long)p.B * p.G * N * p.L;

  for (int k = max(first, end); k < last; ++k) {  // behind the row's end
    const int t0 = k * TB + tl * 8;
    float o[8] = {};
    if (live && t0 < p.L) {
      store8((T*)q.du + row * p.L, t0, p.L, n, p.out_vec, o);
      store8((T*)q.ddelta + row * p.L, t0, p.L, n, p.out_vec, o);
      if (z) store8((T*)q.dz + row * p.L, t0, p.L, n, p.out_vec, o);
    }
    for (int i = tid; i < N * TB; i += kThreads) {
      const int t = k * TB + i % TB;
      if (t < p.L) {
        pbc[(long long)(i / TB) * p.L + t] = 0.f;
        pbc[pstep + (long long)(i / TB) * p.L + t] = 0.f;
      }
    }
  }

  auto fetch = [&](int k) {
    const int t0 = k * TB + tl * 8, m = live ? n : 0;
    fetch8(sm.in[k & 1][0][tid], u, t0, p.L, m, p.u.vec);
    fetch8(sm.in[k & 1][1][tid], delta, t0, p.L, m, p.delta.vec);
    fetch8(sm.in[k & 1][2][tid], dy, t0, p.L, m, p.dy.vec);
    if (z) fetch8(sm.in[k & 1][3][tid], z, t0, p.L, m, p.z.vec);
  };
  constexpr int kRow = TB / 8, kPer = kStates * kRow * 2 / kThreads;
  static_assert(kStates * kRow * 2 % kThreads == 0 && kStates * CH == kThreads, "whole vectors and words a thread");
  // B, C and entering states of chunk ch of block k, the it-th in order
  auto fetch_tile = [&](int k, int ch, int it) {
    const int s0 = ch * kStates;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = tid + j * kThreads, s = s0 + v / kRow % kStates, t0 = k * TB + v % kRow * 8;
      const bool second = v >= kStates * kRow;
      if (s < N)
        fetch8(sm.raw[j][tid], (second ? Ct : Bt) + s * (second ? p.Ct.rs : p.Bt.rs), t0, p.L, n,
               second ? p.Ct.vec : p.Bt.vec);
    }
    const int s = s0 + tid % kStates, cc = tid / kStates;
    float* d = &sm.ck[it & 1][tid % kStates][cc];
    if (s < N && tile * CH + cc < E)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(shared_addr(d)),
                   "l"(q.ckpt + (((long long)b * p.H + g * E + tile * CH + cc) * nck + k) * N + s)
                   : "memory");
    else
      *d = 0.f;
  };
  auto commit_tile = [&](int k, int ch, int it) {
    fetched();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = tid + j * kThreads, s = v / kRow % kStates, t = v % kRow * 8;
      float w[8] = {};
      if (ch * kStates + s < N) take8(sm.raw[j][tid], k * TB + t, n, w);
      float* d = sm.tile[it & 1][v >= kStates * kRow][s];
      *reinterpret_cast<float4*>(d + tile_at(t)) = make_float4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<float4*>(d + tile_at(t + 4)) = make_float4(w[4], w[5], w[6], w[7]);
    }
  };
  if (first < end) {
    fetch(end - 1);
    fetch_tile(end - 1, 0, 0);
    commit_tile(end - 1, 0, 0);
  }
  __syncthreads();
  float sum_d = 0.f, sum_bias = 0.f;
  int it = 0;
  for (int k = end - 1; k >= first; --k) {
    const int t0 = k * TB + tl * 8, m = live ? n : 0;
    float2 dt[PAIRS], du[PAIRS], dyp[PAIRS], gB[PAIRS], gA[PAIRS], y0[PAIRS];
    float sum;
    {
      float v[8], d[8], e[8];
      take8(sm.in[k & 1][0][tid], t0, m, v);
      take8(sm.in[k & 1][1][tid], t0, INT_MAX, d);
      take8(sm.in[k & 1][2][tid], t0, m, e);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) dt[i] = add2(make_float2(d[2 * i], d[2 * i + 1]), both(bias));
      if (p.softplus) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) dt[i] = softplus2(dt[i]);
      }
      if (t0 + 8 > n) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          if (t0 + 2 * i >= n) dt[i].x = 0.f;
          if (t0 + 2 * i + 1 >= n) dt[i].y = 0.f;
        }
      }
      const float2 s2 = add2(add2(dt[0], dt[1]), add2(dt[2], dt[3]));
      sum = s2.x + s2.y;
      if (z) {
        take8(sm.in[k & 1][3][tid], t0, m, d);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const float2 g2 = mul2(pair(e, i), silu2(pair(d, i)));
          e[2 * i] = g2.x;
          e[2 * i + 1] = g2.y;
        }
      }
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float2 uv = make_float2(v[2 * i], v[2 * i + 1]);
        du[i] = mul2(dt[i], uv);
        y0[i] = mul2(both(Dh), uv);
        dyp[i] = make_float2(e[2 * i], e[2 * i + 1]);
        gB[i] = gA[i] = make_float2(0.f, 0.f);
      }
    }
    if (k > first) fetch(k - 1);
    for (int ch = 0; ch < chunks; ++ch, ++it) {
      const int s0 = ch * kStates, ns = min(N - s0, kStates);
      const bool more = ch + 1 < chunks || k > first;
      const int kn = ch + 1 < chunks ? k : k - 1, cn = ch + 1 < chunks ? ch + 1 : 0;
      if (more) fetch_tile(kn, cn, it + 1);
      const float* xin = tl == 0 ? &sm.ck[it & 1][0][c] : &sm.zero[0][c];
      const float* rin = tl == TL - 1 ? gs + s0 * CH + c : &sm.zero[0][c];
#pragma unroll 1
      for (int s = 0; s < ns; ++s) {
        const float An = As[(s0 + s) * CH + c], A2 = An * kLog2e, x0 = xin[s * CH], r0 = rin[s * CH];
        const float4* Bp = reinterpret_cast<const float4*>(sm.tile[it & 1][0][s]) + tl;
        const float4* Cp = reinterpret_cast<const float4*>(sm.tile[it & 1][1][s]) + tl;
        const float4 b0 = Bp[0], b1 = Bp[TL], c0 = Cp[0], c1 = Cp[TL];
        const float2 Bv[PAIRS] = {{b0.x, b0.y}, {b0.z, b0.w}, {b1.x, b1.y}, {b1.z, b1.w}};
        const float2 Cv[PAIRS] = {{c0.x, c0.y}, {c0.z, c0.w}, {c1.x, c1.y}, {c1.z, c1.w}};
        float2 a[PAIRS], w[PAIRS], cy[PAIRS], ax[PAIRS];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const float2 e = mul2(dt[i], both(A2));
          a[i] = make_float2(ex2(e.x), ex2(e.y));
          w[i] = mul2(du[i], Bv[i]);
          cy[i] = mul2(Cv[i], dyp[i]);
        }
        // both recurrences from zero: hf is the state at the lane's end, hb what its first step hands on
        float Pf = ex2(sum * A2), Pb = Pf;
        float hf = fmaf(a[0].y, w[0].x, w[0].y);
#pragma unroll
        for (int i = 1; i < PAIRS; ++i) {
          hf = fmaf(a[i].x, hf, w[i].x);
          hf = fmaf(a[i].y, hf, w[i].y);
        }
        float2 ac = mul2(a[PAIRS - 1], cy[PAIRS - 1]);
        float hb = fmaf(a[PAIRS - 1].x, ac.y, ac.x);
#pragma unroll
        for (int i = PAIRS - 2; i >= 0; --i) {
          ac = mul2(a[i], cy[i]);
          hb = fmaf(a[i].y, hb, ac.y);
          hb = fmaf(a[i].x, hb, ac.x);
        }
        hf = fmaf(Pf, x0, hf);
        hb = fmaf(Pb, r0, hb);
        join<true, 1>(hf, Pf);
        join<false, 1>(hb, Pb);
        join<true, 2>(hf, Pf);
        join<false, 2>(hb, Pb);
        join<true, 4>(hf, Pf);
        join<false, 4>(hb, Pb);
        put_shared(r1s + (s0 + s) * CH * 4, hb);
        float x = neighbour<true>(hf, x0), r = neighbour<false>(hb, r0);
        float2 v[PAIRS];  // dC, then dB of the channel
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          ax[i].x = a[i].x * x;
          float2 xv;
          xv.x = x = ax[i].x + w[i].x;
          ax[i].y = a[i].y * x;
          xv.y = x = ax[i].y + w[i].y;
          y0[i] = fma2(Cv[i], xv, y0[i]);
          v[i] = mul2(dyp[i], xv);
        }
        float* out = sm.sums[warp][s][0] + tl * 8 + cl * 2;
        *reinterpret_cast<float2*>(out + TB) = sum_channels(v, cl);
        float2 da = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = PAIRS - 1; i >= 0; --i) {
          float2 gg;
          gg.y = cy[i].y + r;
          r = a[i].y * gg.y;
          gg.x = cy[i].x + r;
          r = a[i].x * gg.x;
          gB[i] = fma2(gg, Bv[i], gB[i]);
          const float2 mm = mul2(gg, ax[i]);
          v[i] = mul2(gg, du[i]);
          gA[i] = fma2(both(An), mm, gA[i]);
          da = fma2(dt[i], mm, da);
        }
        *reinterpret_cast<float2*>(out) = sum_channels(v, cl);
        float d = da.x + da.y;
        if (!lanes) {
#pragma unroll
          for (int e = CL; e < 32; e *= 2) d += __shfl_xor_sync(~0u, d, e);
        }
        da_at[(s0 + s) * da_step] += d;
      }
      if (more) commit_tile(kn, cn, it + 1);
      __syncthreads();
      for (int i = tid; i < ns * 2 * (TB / 4); i += kThreads) {  // four steps of dB or dC of a state
        const float4* q = reinterpret_cast<const float4*>(&sm.sums[0][0][0][0]) + i;
        constexpr int kWarp4 = kStates * 2 * TB / 4;
        float4 v = q[0];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 o = q[w * kWarp4];
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        const int t = k * TB + i % (TB / 4) * 4, row = i / (TB / 4);
        float* o = pbc + (row & 1) * pstep + (long long)(s0 + row / 2) * p.L + t;
        if (p.L % 4 == 0) {
          if (t < p.L) *reinterpret_cast<float4*>(o) = v;
        } else {
          if (t < p.L) o[0] = v.x;
          if (t + 1 < p.L) o[1] = v.y;
          if (t + 2 < p.L) o[2] = v.z;
          if (t + 3 < p.L) o[3] = v.w;
        }
      }
      __syncthreads();
    }
    if (live && t0 < p.L) {
      float v[8], o[8], w[8];
      take8(sm.in[k & 1][0][tid], t0, n, v);
      float2 sd = make_float2(0.f, 0.f), sb = sd;
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        const float2 g2 = fma2(dt[i], gB[i], mul2(both(Dh), dyp[i]));
        o[2 * i] = g2.x;
        o[2 * i + 1] = g2.y;
        sd = fma2(dyp[i], pair(v, i), sd);
      }
      sum_d += sd.x + sd.y;
      store8((T*)q.du + row * p.L, t0, p.L, n, p.out_vec, o);
      take8(sm.in[k & 1][1][tid], t0, n, w);
#pragma unroll
      for (int i = 0; i < PAIRS; ++i) {
        float2 g2 = fma2(pair(v, i), gB[i], gA[i]);
        if (p.softplus) g2 = mul2(g2, sigmoid2(add2(pair(w, i), both(bias))));
        if (t0 + 2 * i >= n) g2.x = 0.f;
        if (t0 + 2 * i + 1 >= n) g2.y = 0.f;
        sb = add2(sb, g2);
        o[2 * i] = g2.x;
        o[2 * i + 1] = g2.y;
      }
      sum_bias += sb.x + sb.y;
      store8((T*)q.ddelta + row * p.L, t0, p.L, n, p.out_vec, o);
      if (z) {
        take8(sm.in[k & 1][2][tid], t0, n, v);
        take8(sm.in[k & 1][3][tid], t0, n, w);
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
          const float2 g2 = mul2(mul2(pair(v, i), y0[i]), dsilu2(pair(w, i)));
          o[2 * i] = g2.x;
          o[2 * i + 1] = g2.y;
        }
        store8((T*)q.dz + row * p.L, t0, p.L, n, p.out_vec, o);
      }
    }
  }
#pragma unroll
  for (int d = CL; d < 32; d *= 2) {
    sum_d += __shfl_xor_sync(~0u, sum_d, d);
    sum_bias += __shfl_xor_sync(~0u, sum_bias, d);
  }
  const long long part = (long long)b * sg.count + seg;
  if (live && tl == 0) {
    q.part_d[part * p.H + h] = sum_d;
    q.part_d[((long long)p.B * sg.count + part) * p.H + h] = sum_bias;
  }
  __syncthreads();
  for (int i = tid; i < N * CH; i += kThreads) {
    const int cc = i / N, s = i % N, hh = g * E + tile * CH + cc;
    if (tile * CH + cc >= E) continue;
    float v = 0.f;
    if (lanes) {
#pragma unroll
      for (int j = 0; j < TL; ++j) v += das[s * kThreads + cc / CL * 32 + j * CL + cc % CL];
    } else {
      v = das[s * CH + cc];
    }
    q.part_a[(part * p.H + hh) * N + s] = v;
    if (q.dstate_in && seg == 0) q.dstate_in[((long long)b * p.H + hh) * N + s] = gs[s * CH + cc];
  }
}

// dB and dC: the blocks' parts, in order.
template <typename T>
__global__ void scan_sum_bc_kernel(const float* part, T* dB, T* dC, long long m, int tiles) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= 2 * m) return;
  float v = 0.f;
  for (int k = 0; k < tiles; ++k) v += part[k * 2 * m + i];
  if (i < m)
    IO<T>::st(dB + i, v);
  else
    IO<T>::st(dC + (i - m), v);
}

// dA, dD and ddt_bias: the batch rows' parts, in order.
__global__ void scan_sum_rows_kernel(const float* part_a, const float* part_d, float* dA, float* dD, float* dbias,
                                     int B, long long H, int N) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long m = H * N;
  if (i >= m + 2 * H) return;
  const float* src = i < m ? part_a + i : part_d + (i < m + H ? i - m : B * H + i - m - H);
  const long long stride = i < m ? m : H;
  float v = 0.f;
  for (int b = 0; b < B; ++b) v += src[b * stride];
  if (i < m)
    dA[i] = v;
  else if (i < m + H) {
    if (dD) dD[i - m] = v;
  } else if (dbias) {
    dbias[i - m - H] = v;
  }
}

struct Plan {
  int tiles;
  Segments sg;
  size_t bc, a, d;  // bytes of the parts
};
Plan plan(int B, int H, int L, int N, int G) {
  const int tiles = (H / G + CH - 1) / CH, all = (L + TB - 1) / TB, sms = num_sms();
  const long long ctas = (long long)tiles * B * G;
  Plan r{tiles, {1, all, nullptr, nullptr}, 0, 0, 0};
  float least = -1.f;
  for (int want = 1; want <= 64 && (want == 1 || ctas * (want - 1) < 16 * sms); ++want) {
    const int blocks = (all + want - 1) / want, count = (all + blocks - 1) / blocks;
    if (count != want || (count > 1 && blocks < 4)) continue;
    // measured: 130 us and 80 us for each thread block on an SM, 2048 steps of 16 states in bf16
    const float t = scan_cost(ctas * count, blocks, kMinBlocks, 130.f, 80.f, sms) +
                    (count > 1 ? ends_cost(B, H, G, N, count, blocks, sms) : 0.f);
    if (least < 0.f || t < least) {
      least = t;
      r.sg = {count, blocks, nullptr, nullptr};
    }
  }
  r.bc = up256((size_t)tiles * 2 * B * G * N * L * 4);
  r.a = up256((size_t)B * r.sg.count * H * N * 4);
  r.d = up256((size_t)2 * B * r.sg.count * H * 4);
  return r;
}

template <typename T>
cudaError_t bwd(const ScanArgs& p, BwdOut q, void* dB, void* dC, float* dA, float* dD, float* dbias, char* ws,
                int dtype, cudaStream_t st) {
  Plan pl = plan(p.B, p.H, p.L, p.N, p.G);
  q.part_bc = (float*)ws;
  q.part_a = (float*)(ws + pl.bc);
  q.part_d = (float*)(ws + pl.bc + pl.a);
  place_segments(&pl.sg, ws + pl.bc + pl.a + pl.d, p.B, p.H, p.N);
  cudaError_t e;
  if (pl.sg.count > 1 && (e = launch_segment_states(p, pl.sg, q.dstate_out, true, dtype, st)) != cudaSuccess) return e;
  const int Np = (p.N + kStates - 1) / kStates * kStates;
  const size_t smem = sizeof(Sm<T>) + (size_t)Np * (3 * CH + (Np <= kLaneStates ? kThreads : 2 * CH)) * 4;
  e = smem_optin<scan_bwd_kernel<T>>(smem);
  if (e != cudaSuccess) return e;
  scan_bwd_kernel<T><<<(unsigned)((long long)pl.tiles * p.B * p.G * pl.sg.count), kThreads, smem, st>>>(p, q, pl.sg,
                                                                                                      pl.tiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long m = (long long)p.B * p.G * p.N * p.L, r = (long long)p.H * (p.N + 2);
  scan_sum_bc_kernel<T><<<(unsigned)((2 * m + 255) / 256), 256, 0, st>>>(q.part_bc, (T*)dB, (T*)dC, m, pl.tiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  scan_sum_rows_kernel<<<(unsigned)((r + 255) / 256), 256, 0, st>>>(q.part_a, q.part_d, dA, dD, dbias,
                                                                    p.B * pl.sg.count, p.H, p.N);
  return cudaGetLastError();
}

}  // namespace

size_t selective_scan_bwd_workspace_bytes(int B, int H, int L, int N, int G) {
  const Plan pl = plan(B, H, L, N, G);
  return pl.bc + pl.a + pl.d + segments_bytes(pl.sg, B, H, N);
}

cudaError_t launch_selective_scan_bwd(const ScanArgs& p, const float* ckpt, void* du, void* ddelta, float* dA, void* dB,
                                      void* dC, float* dD, float* ddt_bias, void* dz, const float* dstate_out,
                                      float* dstate_in, void* workspace, int dtype, cudaStream_t st) {
  const BwdOut q{du, ddelta, dz, ckpt, dstate_out, dstate_in, nullptr, nullptr, nullptr};
  switch (dtype) {
    case 0: return bwd<float>(p, q, dB, dC, dA, dD, ddt_bias, (char*)workspace, dtype, st);
    case 1: return bwd<__half>(p, q, dB, dC, dA, dD, ddt_bias, (char*)workspace, dtype, st);
    case 2: return bwd<__nv_bfloat16>(p, q, dB, dC, dA, dD, ddt_bias, (char*)workspace, dtype, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fc
