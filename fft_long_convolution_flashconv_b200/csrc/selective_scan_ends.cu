// States entering the segments of a long selective scan, forward and backward.
//
// What a segment leaves behind without an entering state is a plain weighted
// sum, with no recurrence:
//   forward, at its end:     sum_t exp(A (S_end - S_t)) dt_t B_t u_t
//   backward, at its start:  sum_t exp(A (S_t - S_start)) C_t dyp_t
// with S the running sum of dt (including step t).  So a lane runs through its
// steps with the sum of dt between them and the segment's edge, and only those
// sums pass between lanes, once a block and not once a state.  One exponential,
// a product for its argument, one with B or C and a multiply-add a state and
// step: bound by the special function unit, 9.85 cycles a warp, state and step
// where its floor is 8 (151 us for 15 of 16 segments of 4 x 1024 channels of 8192
// steps, 16 states, bf16).
#include "kernels.cuh"
#include "scan.cuh"

namespace fc {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kStates = 16;  // states of a block, in registers
constexpr int TPL = 16, TL = kCkptSteps / TPL, CL = 32 / TL, CH = kWarps * CL, TB = kCkptSteps;
constexpr int PAIRS = TPL / 2, VPL = TPL / kVec;

template <typename T>
struct Sm {
  T in[2][3][VPL][kThreads][8];           // u and delta, or delta, dy and z, of even and odd blocks
  T raw[kStates * TB / 8 / kThreads][kThreads][8];  // B or C on its way
  float tile[2][kStates][TB];             // as floats: lane by lane in quarters (tile_at)
};

__device__ __forceinline__ int tile_at(int t) { return (t % TPL / 4) * (TL * 4) + t / TPL * 4 + t % 4; }

template <typename T, bool BACK>
__global__ __launch_bounds__(kThreads, 4) void scan_ends_kernel(ScanArgs p, Segments sg, int tiles, int chunks) {
  extern __shared__ float4 smem4[];
  Sm<T>& sm = *reinterpret_cast<Sm<T>*>(smem4);
  const int tid = threadIdx.x, lane = tid & 31, tl = lane % TL, c = (tid >> 5) * CL + lane / TL, N = p.N;
  // the last segment's end (backward: the first one's start) enters no segment
  int i = blockIdx.x;
  const int seg = i % (sg.count - 1) + (BACK ? 1 : 0);
  i /= sg.count - 1;
  const int s0 = i % chunks * kStates, ns = min(N - s0, kStates);
  i /= chunks;
  const int tile = i % tiles, bg = i / tiles, b = bg / p.G, g = bg % p.G, E = p.H / p.G;
  const int n = row_length(p.lengths, b, p.L);
  const bool live = tile * CH + c < E;
  const int h = g * E + (live ? tile * CH + c : 0);
  const long long row = (long long)b * p.H + h;
  const float bias = p.dt_bias ? __ldg(p.dt_bias + h) : 0.f;
  const T* u = (const T*)p.u.p + b * p.u.bs + h * p.u.rs;
  const T* delta = (const T*)p.delta.p + b * p.delta.bs + h * p.delta.rs;
  const T* z = p.z.p ? (const T*)p.z.p + b * p.z.bs + h * p.z.rs : nullptr;
  const T* dy = BACK ? (const T*)p.dy.p + b * p.dy.bs + h * p.dy.rs : nullptr;
  const Rows& br = BACK ? p.Ct : p.Bt;
  const T* bt = (const T*)br.p + b * br.bs + g * br.gs + s0 * br.rs;
  const int first = seg * sg.blocks, end = min(min((p.L + TB - 1) / TB, first + sg.blocks), (n + TB - 1) / TB);
  float A2[kStates];
  float2 acc[kStates];
#pragma unroll
  for (int s = 0; s < kStates; ++s) {
    A2[s] = live && s < ns ? __ldg(p.A + (long long)h * N + s0 + s) * kLog2e : 0.f;
    acc[s] = make_float2(0.f, 0.f);
  }
  constexpr int kPer = kStates * TB / 8 / kThreads, kRow = TB / 8;
  // blocks in the order of growing distance from the edge
  auto at = [&](int k) { return BACK ? first + k : end - 1 - k; };
  auto fetch = [&](int k) {
    const int tb = at(k) * TB;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int t0 = tb + tl * TPL + j * 8;
      if (BACK) {
        fetch8(sm.in[k & 1][0][j][tid], dy, t0, p.L, n, p.dy.vec);
        if (z) fetch8(sm.in[k & 1][2][j][tid], z, t0, p.L, n, p.z.vec);
      } else {
        fetch8(sm.in[k & 1][0][j][tid], u, t0, p.L, n, p.u.vec);
      }
      fetch8(sm.in[k & 1][1][j][tid], delta, t0, p.L, n, p.delta.vec);
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = tid + j * kThreads, s = v / kRow;
      if (s < ns) fetch8(sm.raw[j][tid], bt + s * br.rs, tb + v % kRow * 8, p.L, n, br.vec);
    }
  };
  auto commit = [&](int k) {
    const int tb = at(k) * TB;
    fetched();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = tid + j * kThreads, s = v / kRow, t = v % kRow * 8;
      float w[8] = {};
      if (s < ns) take8(sm.raw[j][tid], tb + t, n, w);
      float* d = sm.tile[k & 1][s];
      *reinterpret_cast<float4*>(d + tile_at(t)) = make_float4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<float4*>(d + tile_at(t + 4)) = make_float4(w[4], w[5], w[6], w[7]);
    }
  };
  const int blocks = end - first;
  float edge = 0.f;  // sum of dt between the edge and the block
  if (blocks > 0) {
    fetch(0);
    commit(0);
  }
  __syncthreads();
  for (int k = 0; k < blocks; ++k) {
    float2 S[PAIRS], w[PAIRS];
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int t0 = at(k) * TB + tl * TPL + j * 8;
      float v[8], d[8];
      take8(sm.in[k & 1][1][j][tid], t0, INT_MAX, d);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 x = add2(make_float2(d[2 * e], d[2 * e + 1]), both(bias));
        if (p.softplus) x = softplus2(x);
        if (t0 + 2 * e >= n) x.x = 0.f;
        if (t0 + 2 * e + 1 >= n) x.y = 0.f;
        S[4 * j + e] = x;
      }
      take8(sm.in[k & 1][0][j][tid], t0, n, v);
      if (BACK) {
        if (z) {
          float zv[8];
          take8(sm.in[k & 1][2][j][tid], t0, n, zv);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= silu(zv[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * j + e] = make_float2(v[2 * e], v[2 * e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * j + e] = mul2(S[4 * j + e], make_float2(v[2 * e], v[2 * e + 1]));
      }
    }
    if (k + 1 < blocks) fetch(k + 1);  // this thread is done with the other buffer's values
    // running sums towards the edge: inclusive of the step backward, exclusive forward
#pragma unroll
    for (int e = 0; e < TPL; ++e) {
      const int i2 = BACK ? e : TPL - 1 - e;
      float& v = i2 & 1 ? S[i2 / 2].y : S[i2 / 2].x;
      const float d = v;
      if (BACK) {
        sum += d;
        v = sum;
      } else {
        v = sum;
        sum += d;
      }
    }
    float scan = sum;
#pragma unroll
    for (int d = 1; d < TL; d *= 2) {
      const float o = BACK ? __shfl_up_sync(~0u, scan, d, TL) : __shfl_down_sync(~0u, scan, d, TL);
      if (BACK ? tl >= d : tl + d < TL) scan += o;
    }
    // the lanes between this one and the edge: taken from the neighbour, since scan - sum would cancel away small
    // distances behind one large step
    const float ahead = BACK ? __shfl_up_sync(~0u, scan, 1, TL) : __shfl_down_sync(~0u, scan, 1, TL);
    const float off = edge + (tl == (BACK ? 0 : TL - 1) ? 0.f : ahead);
    edge += __shfl_sync(~0u, scan, BACK ? TL - 1 : 0, TL);
#pragma unroll
    for (int e = 0; e < PAIRS; ++e) S[e] = add2(S[e], both(off));
#pragma unroll
    for (int s = 0; s < kStates; ++s) {
      const float4* t = reinterpret_cast<const float4*>(sm.tile[k & 1][s]) + tl;
#pragma unroll
      for (int e = 0; e < TPL / 4; ++e) {
        const float4 bv = t[e * TL];
        const float2 x = mul2(S[2 * e], both(A2[s])), y = mul2(S[2 * e + 1], both(A2[s]));
        acc[s] = fma2(make_float2(ex2(x.x), ex2(x.y)), mul2(w[2 * e], make_float2(bv.x, bv.y)), acc[s]);
        acc[s] = fma2(make_float2(ex2(y.x), ex2(y.y)), mul2(w[2 * e + 1], make_float2(bv.z, bv.w)), acc[s]);
      }
    }
    if (k + 1 < blocks) commit(k + 1);
    __syncthreads();
  }
#pragma unroll
  for (int s = 0; s < kStates; ++s) {
    float v = acc[s].x + acc[s].y;
#pragma unroll
    for (int d = 1; d < TL; d *= 2) v += __shfl_xor_sync(~0u, v, d);
    if (live && s < ns && tl == s % TL) sg.state[(row * sg.count + seg) * N + s0 + s] = v;
  }
  if (live && tl == 0 && s0 == 0) sg.dt[row * sg.count + seg] = edge;
}

// The states entering the segments of a row, in place: x passes a segment as exp(A dt) x + what the segment leaves.
template <bool BACK>
__global__ void join_segments_kernel(Segments sg, const float* A, const float* outer, long long rows, int H, int N) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= rows * N) return;
  const long long row = i / N;
  const int s = (int)(i % N);
  const float A2 = __ldg(A + row % H * N + s) * kLog2e;
  float x = outer ? __ldg(outer + i) : 0.f;
  // eight segments' loads at a time, ahead of the chain
  for (int k = 0; k < sg.count; k += 8) {
    float e[8], d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool on = k + j + 1 < sg.count;
      const int seg = BACK ? sg.count - 1 - k - j : k + j;
      e[j] = on ? sg.state[(row * sg.count + seg) * N + s] : 0.f;
      d[j] = on ? sg.dt[row * sg.count + seg] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (k + j < sg.count) sg.state[(row * sg.count + (BACK ? sg.count - 1 - k - j : k + j)) * N + s] = x;
      x = fmaf(ex2(d[j] * A2), x, e[j]);
    }
  }
}

template <typename T, bool BACK>
cudaError_t run(const ScanArgs& p, const Segments& sg, const float* outer, cudaStream_t st) {
  const int tiles = (p.H / p.G + CH - 1) / CH, chunks = (p.N + kStates - 1) / kStates;
  cudaError_t e = smem_optin<scan_ends_kernel<T, BACK>>(sizeof(Sm<T>));
  if (e != cudaSuccess) return e;
  const long long grid = (long long)tiles * p.B * p.G * (sg.count - 1) * chunks, rows = (long long)p.B * p.H;
  scan_ends_kernel<T, BACK><<<(unsigned)grid, kThreads, sizeof(Sm<T>), st>>>(p, sg, tiles, chunks);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  join_segments_kernel<BACK><<<(unsigned)((rows * p.N + 127) / 128), 128, 0, st>>>(sg, p.A, outer, rows, p.H, p.N);
  return cudaGetLastError();
}
template <typename T>
cudaError_t run(const ScanArgs& p, const Segments& sg, const float* outer, bool back, cudaStream_t st) {
  return back ? run<T, true>(p, sg, outer, st) : run<T, false>(p, sg, outer, st);
}

}  // namespace

cudaError_t launch_segment_states(const ScanArgs& p, const Segments& sg, const float* outer, bool back, int dtype,
                                  cudaStream_t st) {
  switch (dtype) {
    case 0: return run<float>(p, sg, outer, back, st);
    case 1: return run<__half>(p, sg, outer, back, st);
    case 2: return run<__nv_bfloat16>(p, sg, outer, back, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fc
