// Backward pass of the selective scan.
//
// With dyp = dy silu(z) and the adjoint g_n[t] = C_n[t] dyp[t] + a_n[t+1] g_n[t+1]
// of the state x_n[t]:
//   du = D dyp + dt sum_n g_n B_n
//   ddt = u sum_n g_n B_n + sum_n A_n g_n a_n x_n[t-1],  ddelta = ddt softplus'
//   dA_n = sum_{b,t} dt g_n a_n x_n[t-1],  dD = sum dyp u,  ddt_bias = sum ddelta
//   dB_n[t] = sum_h g_n dt u,  dC_n[t] = sum_h dyp x_n,  dz = dy y silu'(z)
//
// A warp takes four channels by 64 steps (eight lanes of eight steps a
// channel) and walks through the 64-step blocks from the last to the first.
// In a block it runs each state forward again from the kept state that enters
// the block, then its adjoint backward; both recurrences are joined over a
// channel's lanes by shuffles.  dB and dC are summed over the warp's channels
// by shuffles, over the block's warps in shared memory and over the blocks by
// scan_sum_kernel, always in the same order, so results do not change from
// run to run.
#include "kernels.cuh"
#include "scan.cuh"

namespace fc {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kStates = 16;  // states whose tiles are in shared memory at a time
constexpr int TL = 8, CL = 4, TB = kCkptSteps, CH = kWarps * CL;
static_assert(TB == TL * 8, "a block of steps is what a channel's lanes hold");

struct BwdOut {
  void *du, *ddelta, *dz;
  const float* ckpt;
  const float* dstate_out;
  float* dstate_in;
  float* part_bc;  // [tiles][2][B][G][N][L]
  float* part_a;   // [B][H][N]
  float* part_d;   // [B][H] dD, then [B][H] ddt_bias
};

// Sum v over the four lanes lane ^ 8, lane ^ 16: lane (cl, tl) returns the sums
// of elements 2 cl and 2 cl + 1 of the eight.
__device__ __forceinline__ float2 sum_channels(const float (&v)[8], int cl) {
  float w[4];
  const bool hi = cl & 2, odd = cl & 1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float give = hi ? v[i] : v[i + 4], keep = hi ? v[i + 4] : v[i];
    w[i] = keep + __shfl_xor_sync(~0u, give, 16);
  }
  float r[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float give = odd ? w[i] : w[i + 2], keep = odd ? w[i + 2] : w[i];
    r[i] = keep + __shfl_xor_sync(~0u, give, 8);
  }
  return make_float2(r[0], r[1]);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void scan_bwd_kernel(ScanArgs p, BwdOut q, int tiles) {
  extern __shared__ float4 smem4[];
  float* Bs = reinterpret_cast<float*>(smem4);  // [kStates][TB]
  float* Cs = Bs + kStates * TB;
  float* wb = Cs + kStates * TB;                    // [kWarps][kStates][2][TB] dB, dC of a warp's channels
  float* As = wb + kWarps * kStates * 2 * TB;       // [N][CH]
  float* gs = As + p.N * CH;                        // [N][CH] a g of the first step behind the block
  float* das = gs + p.N * CH;                       // [N][CH] dA
  const int tid = threadIdx.x, lane = tid & 31, tl = lane % TL, cl = lane / TL, warp = tid >> 5;
  const int c = warp * CL + cl;
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
    As[i] = ok ? __ldg(p.A + (long long)hh * N + s) : 0.f;
    gs[i] = ok && q.dstate_out ? __ldg(q.dstate_out + ((long long)b * p.H + hh) * N + s) : 0.f;
    das[i] = 0.f;
  }
  const T* u = (const T*)p.u.p + b * p.u.bs + h * p.u.rs;
  const T* delta = (const T*)p.delta.p + b * p.delta.bs + h * p.delta.rs;
  const T* dy = (const T*)p.dy.p + b * p.dy.bs + h * p.dy.rs;
  const T* z = p.z.p ? (const T*)p.z.p + b * p.z.bs + h * p.z.rs : nullptr;
  const T* Bt = (const T*)p.Bt.p + b * p.Bt.bs + g * p.Bt.gs;
  const T* Ct = (const T*)p.Ct.p + b * p.Ct.bs + g * p.Ct.gs;
  const float Dh = p.D ? __ldg(p.D + h) : 0.f, bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
  const int nck = (p.L + TB - 1) / TB;
  float* pbc = q.part_bc + ((long long)tile * 2 * p.B * p.G + bg) * N * p.L;  // dB; dC is B G N L further
  const long long pstep = (long long)p.B * p.G * N * p.L;
  float sum_d = 0.f, sum_bias = 0.f;
  for (int k = nck - 1; k >= 0; --k) {
    const int tb = k * TB, t0 = tb + tl * 8;
    if (tb >= n) {
      float o[8] = {};
      if (live && t0 < p.L) {
        store8((T*)q.du + row * p.L, t0, p.L, n, p.out_vec, o);
        store8((T*)q.ddelta + row * p.L, t0, p.L, n, p.out_vec, o);
        if (z) store8((T*)q.dz + row * p.L, t0, p.L, n, p.out_vec, o);
      }
      for (int i = tid; i < N * TB; i += kThreads) {
        const int t = tb + i % TB;
        if (t < p.L) {
          pbc[(long long)(i / TB) * p.L + t] = 0.f;
          pbc[pstep + (long long)(i / TB) * p.L + t] = 0.f;
        }
      }
      continue;
    }
    float dt[8], du[8], dyp[8], gB[8], gA[8], y0[8], sum = 0.f;
    {
      float v[8];
      load8(u, t0, p.L, live ? n : 0, p.u.vec, v);
      load8(delta, t0, p.L, n, p.delta.vec, dt);
      load8(dy, t0, p.L, live ? n : 0, p.dy.vec, dyp);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float r = dt[i] + bias;
        dt[i] = t0 + i < n ? (p.softplus ? softplus(r) : r) : 0.f;
        sum += dt[i];
        du[i] = dt[i] * v[i];
        y0[i] = Dh * v[i];
        gB[i] = gA[i] = 0.f;
      }
      if (z) {
        load8(z, t0, p.L, n, p.z.vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) dyp[i] *= silu(v[i]);
      }
    }
    for (int s0 = 0; s0 < N; s0 += kStates) {
      const int ns = min(kStates, N - s0);
      __syncthreads();
      for (int i = tid; i < ns * TL; i += kThreads) {
        const int s = i / TL, j = i % TL;
        float w[8];
        load8(Bt + (s0 + s) * p.Bt.rs, tb + j * 8, p.L, n, p.Bt.vec, w);
        float4* d = reinterpret_cast<float4*>(Bs + s * TB);
        d[j] = make_float4(w[0], w[1], w[2], w[3]);
        d[TL + j] = make_float4(w[4], w[5], w[6], w[7]);
        load8(Ct + (s0 + s) * p.Ct.rs, tb + j * 8, p.L, n, p.Ct.vec, w);
        d = reinterpret_cast<float4*>(Cs + s * TB);
        d[j] = make_float4(w[0], w[1], w[2], w[3]);
        d[TL + j] = make_float4(w[4], w[5], w[6], w[7]);
      }
      __syncthreads();
      for (int s = 0; s < ns; ++s) {
        const float An = As[(s0 + s) * CH + c], A2 = An * kLog2e;
        const float4* Bp = reinterpret_cast<const float4*>(Bs + s * TB);
        const float4* Cp = reinterpret_cast<const float4*>(Cs + s * TB);
        const float4 b0 = Bp[tl], b1 = Bp[TL + tl], c0 = Cp[tl], c1 = Cp[TL + tl];
        const float Bv[8] = {b0.x, b0.y, b0.z, b0.w, b1.x, b1.y, b1.z, b1.w};
        const float Cv[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        float a[8], ax[8], r[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = ex2(dt[i] * A2);
        // forward: states from the kept one
        const float P = ex2(sum * A2);
        float hh = du[0] * Bv[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) hh = fmaf(a[i], hh, du[i] * Bv[i]);
        float x0 = 0.f;
        if (tl == 0) {
          x0 = live ? __ldg(q.ckpt + (row * nck + k) * N + s0 + s) : 0.f;
          hh = fmaf(P, x0, hh);
        }
        float Pf = P;
#pragma unroll
        for (int d = 1; d < TL; d *= 2) {
          const float hp = __shfl_up_sync(~0u, hh, d, TL), Pp = __shfl_up_sync(~0u, Pf, d, TL);
          if (tl >= d) {
            hh = fmaf(Pf, hp, hh);
            Pf *= Pp;
          }
        }
        const float up = __shfl_up_sync(~0u, hh, 1, TL);
        float x = tl == 0 ? x0 : up;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          ax[i] = a[i] * x;
          x = fmaf(du[i], Bv[i], ax[i]);
          y0[i] = fmaf(Cv[i], x, y0[i]);
          r[i] = dyp[i] * x;
        }
        const float2 dc = sum_channels(r, cl);
        // backward: r = a g, what a step hands to the one before it
        float rr = 0.f;
#pragma unroll
        for (int i = 7; i >= 0; --i) rr = a[i] * fmaf(Cv[i], dyp[i], rr);
        float r0 = 0.f;
        if (tl == TL - 1) {
          r0 = gs[(s0 + s) * CH + c];
          rr = fmaf(P, r0, rr);
        }
        float Pb = P;
#pragma unroll
        for (int d = 1; d < TL; d *= 2) {
          const float rp = __shfl_down_sync(~0u, rr, d, TL), Pp = __shfl_down_sync(~0u, Pb, d, TL);
          if (tl + d < TL) {
            rr = fmaf(Pb, rp, rr);
            Pb *= Pp;
          }
        }
        const float down = __shfl_down_sync(~0u, rr, 1, TL);
        float gn = tl == TL - 1 ? r0 : down;
        __syncwarp();
        if (tl == 0) gs[(s0 + s) * CH + c] = rr;
        float da = 0.f;
#pragma unroll
        for (int i = 7; i >= 0; --i) {
          const float gg = fmaf(Cv[i], dyp[i], gn);
          gn = a[i] * gg;
          r[i] = gg * du[i];
          gB[i] = fmaf(gg, Bv[i], gB[i]);
          const float m = gg * ax[i];
          gA[i] = fmaf(An, m, gA[i]);
          da = fmaf(dt[i], m, da);
        }
        const float2 db = sum_channels(r, cl);
#pragma unroll
        for (int d = 1; d < TL; d *= 2) da += __shfl_xor_sync(~0u, da, d);
        if (tl == 0) das[(s0 + s) * CH + c] += da;
        float* w = wb + ((warp * kStates + s) * 2) * TB + tl * 8 + cl * 2;
        *reinterpret_cast<float2*>(w) = db;
        *reinterpret_cast<float2*>(w + TB) = dc;
      }
      __syncthreads();
      for (int i = tid; i < ns * 2 * TB; i += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) v += wb[w * kStates * 2 * TB + i];
        const int t = tb + i % TB, s = s0 + i / (2 * TB), which = i / TB & 1;
        if (t < p.L) pbc[which * pstep + (long long)s * p.L + t] = v;
      }
    }
    if (live) {
      float v[8], o[8];
      load8(u, t0, p.L, n, p.u.vec, v);
      if (t0 < p.L) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = fmaf(dt[i], gB[i], Dh * dyp[i]);
          sum_d = fmaf(dyp[i], v[i], sum_d);
        }
        store8((T*)q.du + row * p.L, t0, p.L, n, p.out_vec, o);
        float raw[8];
        load8(delta, t0, p.L, n, p.delta.vec, raw);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[i] = fmaf(v[i], gB[i], gA[i]);
          if (p.softplus) o[i] *= sigmoid(raw[i] + bias);
          if (t0 + i < n) sum_bias += o[i];
        }
        store8((T*)q.ddelta + row * p.L, t0, p.L, n, p.out_vec, o);
        if (z) {
          float dyv[8];
          load8(z, t0, p.L, n, p.z.vec, v);
          load8(dy, t0, p.L, n, p.dy.vec, dyv);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = dyv[i] * y0[i] * dsilu(v[i]);
          store8((T*)q.dz + row * p.L, t0, p.L, n, p.out_vec, o);
        }
      }
    }
  }
#pragma unroll
  for (int d = 1; d < TL; d *= 2) {
    sum_d += __shfl_xor_sync(~0u, sum_d, d);
    sum_bias += __shfl_xor_sync(~0u, sum_bias, d);
  }
  if (live && tl == 0) {
    q.part_d[row] = sum_d;
    q.part_d[(long long)p.B * p.H + row] = sum_bias;
  }
  __syncthreads();
  for (int i = tid; i < N * CH; i += kThreads) {
    const int cc = i / N, s = i % N;
    if (tile * CH + cc >= E) continue;
    const long long at = ((long long)b * p.H + g * E + tile * CH + cc) * N + s;
    q.part_a[at] = das[s * CH + cc];
    if (q.dstate_in) q.dstate_in[at] = gs[s * CH + cc];
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

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct Plan {
  int tiles;
  size_t bc, a, d;  // bytes of the parts
};
Plan plan(int B, int H, int L, int N, int G) {
  const int tiles = (H / G + CH - 1) / CH;
  return {tiles, up256((size_t)tiles * 2 * B * G * N * L * 4), up256((size_t)B * H * N * 4), up256((size_t)2 * B * H * 4)};
}

template <typename T>
cudaError_t bwd(const ScanArgs& p, BwdOut q, void* dB, void* dC, float* dA, float* dD, float* dbias, char* ws,
                cudaStream_t st) {
  const Plan pl = plan(p.B, p.H, p.L, p.N, p.G);
  q.part_bc = (float*)ws;
  q.part_a = (float*)(ws + pl.bc);
  q.part_d = (float*)(ws + pl.bc + pl.a);
  const size_t smem = (size_t)(2 * kStates * TB + kWarps * kStates * 2 * TB + 3 * p.N * CH) * 4;
  cudaError_t e = smem_optin<scan_bwd_kernel<T>>(smem);
  if (e != cudaSuccess) return e;
  scan_bwd_kernel<T><<<(unsigned)((long long)pl.tiles * p.B * p.G), kThreads, smem, st>>>(p, q, pl.tiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const long long m = (long long)p.B * p.G * p.N * p.L, r = (long long)p.H * (p.N + 2);
  scan_sum_bc_kernel<T><<<(unsigned)((2 * m + 255) / 256), 256, 0, st>>>(q.part_bc, (T*)dB, (T*)dC, m, pl.tiles);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  scan_sum_rows_kernel<<<(unsigned)((r + 255) / 256), 256, 0, st>>>(q.part_a, q.part_d, dA, dD, dbias, p.B, p.H, p.N);
  return cudaGetLastError();
}

}  // namespace

size_t selective_scan_bwd_workspace_bytes(int B, int H, int L, int N, int G) {
  const Plan pl = plan(B, H, L, N, G);
  return pl.bc + pl.a + pl.d;
}

cudaError_t launch_selective_scan_bwd(const ScanArgs& p, const float* ckpt, void* du, void* ddelta, float* dA, void* dB,
                                      void* dC, float* dD, float* ddt_bias, void* dz, const float* dstate_out,
                                      float* dstate_in, void* workspace, int dtype, cudaStream_t st) {
  const BwdOut q{du, ddelta, dz, ckpt, dstate_out, dstate_in, nullptr, nullptr, nullptr};
  switch (dtype) {
    case 0: return bwd<float>(p, q, dB, dC, dA, dD, ddt_bias, (char*)workspace, st);
    case 1: return bwd<__half>(p, q, dB, dC, dA, dD, ddt_bias, (char*)workspace, st);
    case 2: return bwd<__nv_bfloat16>(p, q, dB, dC, dA, dD, ddt_bias, (char*)workspace, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fc
