// State space recurrence, gradients. With a_t = exp(u_t A), p = dy silu(z) and e_t the
// gradient of h_t,
//   e_t = C_t p_t + a_{t+1} e_{t+1},   w_t = e_t a_t h_{t-1},   q_t = sum_n B_t e_t,
//   dB_t = sum_d u x e_t,  dC_t = sum_d p h_t,  dx = u q + skip p,  dz = dy (C h + skip x) silu'(z)
//   du = sum_n A w + x q,  ddt = du softplus',  dA = sum_t u w,  dskip = sum_t p x.
//
// Two launches walk the tokens, then one adds partial sums in a fixed order:
// - States, forward in time: the state entering every tile of 16 tokens, from the segment's
//   start on (zero, h0 for the first), and for each segment what it adds to the state and
//   to the gradient that it passes back: sum_t (a_1 ... a_t) C_t p_t, which needs no walk
//   backward.
// - Gradients, tile by tile backward: a tile's states are computed again from its first one,
//   kept every 4 tokens in shared memory, then by 4 tokens in registers with their decays.
// Three exponentials and about 22 multiply-adds for each (token, channel, state) in all:
// bound by the fp32 pipe.
//
// A thread has 4 states of 4 channels, so that the sums over channels (dB, dC) and those over
// states (q, sum A w, C h) each start inside a thread. What is left goes over lanes by
// halves: a lane passes on half of its sums and keeps the other half. Which one is by
// lane, so a lane's registers hold its states in the order n ^ lane (channels alike), and no
// register has to be selected; B and C are in shared memory in all four orders.
#include <type_traits>

#include "state_space.cuh"

namespace gdr {
namespace {

// ------------------------------------------------------------------ states

constexpr int kThreads = 256;
constexpr int kStates = 8;        // states of a thread

template <int N>
struct PreLayout {
  static constexpr int kLanes = N / kStates;
  static constexpr int kChannels = kThreads / kLanes;
  static constexpr int kTile = kSpaceTile;
  static constexpr int kVecs = kTile * kChannels / 8;
  static constexpr int kPer = (kVecs + kThreads - 1) / kThreads;
  static constexpr int kBcVecs = 2 * kTile * N / 8;
  static constexpr int kBcPer = (kBcVecs + kThreads - 1) / kThreads;
};

template <int N>
struct __align__(16) PreShared {
  float u[PreLayout<N>::kTile][PreLayout<N>::kChannels];
  float g[PreLayout<N>::kTile][PreLayout<N>::kChannels];
  float p[PreLayout<N>::kTile][PreLayout<N>::kChannels];
  float bc[2][PreLayout<N>::kTile][N];
  float bias[PreLayout<N>::kChannels];
  unsigned starts[4];
};

// CUT: there are several segments, which need the gradients that they pass back.
template <typename T, int N, bool CUT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
    space_bwd_states_kernel(const SpaceArgs a, const SpaceSplit sp) {
  using L = PreLayout<N>;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  PreShared<N>& sm = *reinterpret_cast<PreShared<N>*>(raw_smem);
  const int tid = threadIdx.x;
  const Channels ch(a, L::kChannels, blockIdx.x);
  const int seg = blockIdx.y, b = blockIdx.z;
  const int t_begin = seg * sp.seg_len, t_end = min(t_begin + sp.seg_len, a.T);
  const long long row0 = static_cast<long long>(b) * a.T;
  const int ci = tid / L::kLanes, c = ch.first + ci, n0 = (tid % L::kLanes) * kStates;
  const bool live = c < ch.end;
  const size_t state = static_cast<size_t>(a.D) * N, own = static_cast<size_t>(c) * N + n0;
  f32x2 A2[kStates / 2], h[kStates / 2], P[kStates / 2], e[kStates / 2];
  float usum = 0.f;
  {
    float A[kStates], v[kStates];
#pragma unroll
    for (int i = 0; i < kStates; ++i) A[i] = v[i] = 0.f;
    if (live) {
      load8(a.A + own, A);
      if (seg == 0 && a.h0) load8(a.h0 + b * state + own, v);
    }
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) {
      A2[i] = pair(A[2 * i] * kLog2e, A[2 * i + 1] * kLog2e);
      h[i] = pair(v[2 * i], v[2 * i + 1]);
      P[i] = pair(1.f, 1.f);
      e[i] = pair(0.f, 0.f);
    }
  }
  for (int i = tid; i < L::kChannels; i += kThreads)
    sm.bias[i] = a.dt_bias && ch.first + i < ch.end ? a.dt_bias[ch.first + i] : 0.f;

  Raw8<T> rx[L::kPer], rdt[L::kPer], rz[L::kPer], ry[L::kPer], rbc[L::kBcPer];
  bool mark = false;
  constexpr int kBc = CUT ? L::kBcVecs : L::kBcVecs / 2;
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kThreads, t = t0 + v / (L::kChannels / 8);
      const int d = ch.first + 8 * (v % (L::kChannels / 8));
      if (v < L::kVecs && t < t_end && d < ch.end) {
        rx[i].load(static_cast<const T*>(a.x) + (row0 + t) * a.xs + d);
        rdt[i].load(static_cast<const T*>(a.dt) + (row0 + t) * a.dts + d);
        if (CUT) {
          ry[i].load(static_cast<const T*>(a.dy) + (row0 + t) * a.D + d);
          if (a.z) rz[i].load(static_cast<const T*>(a.z) + (row0 + t) * a.zs + d);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = t0 + w / (N / 8), n = 8 * (w % (N / 8));
      rbc[i].zero();
      if (v < kBc && t < t_end)
        rbc[i].load((which ? static_cast<const T*>(a.Cm) + (row0 + t) * a.cs
                           : static_cast<const T*>(a.Bm) + (row0 + t) * a.bs) +
                    ch.group * N + n);
    }
    mark = a.starts && tid < L::kTile && t0 + tid < t_end && a.starts[row0 + t0 + tid] != 0;
  };
  auto stage = [&](int t0) {
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kThreads, t = v / (L::kChannels / 8);
      const int d = 8 * (v % (L::kChannels / 8));
      if (v >= L::kVecs) break;
      float x[8], u[8], p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = u[j] = p[j] = 0.f;
      if (t0 + t < t_end && ch.first + d < ch.end) {
        rx[i].get(x);
        rdt[i].get(u);
        float z[8];
        if (CUT) ry[i].get(p);
        if (CUT && a.z) rz[i].get(z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[j] += sm.bias[d + j];
          if (a.softplus) u[j] = softplus(u[j]);
          x[j] *= u[j];
          if (CUT && a.z) p[j] *= silu(z[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<float4*>(&sm.u[t][d + 4 * j]) =
            make_float4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
        *reinterpret_cast<float4*>(&sm.g[t][d + 4 * j]) =
            make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        if (CUT)
          *reinterpret_cast<float4*>(&sm.p[t][d + 4 * j]) =
              make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
      }
    }
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      if (v >= kBc) break;
      float x[8];
      rbc[i].get(x);
      float4* p = reinterpret_cast<float4*>(&sm.bc[which][w / (N / 8)][8 * (w % (N / 8))]);
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    const unsigned m = __ballot_sync(0xffffffffu, mark);
    if (tid == 0) sm.starts[0] = m;
  };
  auto put = [&](float* out, const f32x2 (&v)[kStates / 2]) {
    float f[kStates];
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) split(v[i], f[2 * i], f[2 * i + 1]);
    reinterpret_cast<float4*>(out + own)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(out + own)[1] = make_float4(f[4], f[5], f[6], f[7]);
  };

  bool cleared = false;     // a document starts in what has been walked of the segment
  auto token = [&](int t, bool first) {
    const float u = sm.u[t][ci], g = sm.g[t][ci];
    if (first) {
      cleared = true;
#pragma unroll
      for (int i = 0; i < kStates / 2; ++i) h[i] = P[i] = pair(0.f, 0.f);
    }
    usum += u;
    const f32x2 u2 = pair(u, u), g2 = pair(g, g);
    f32x2 p2;
    if (CUT) {
      const float p = sm.p[t][ci];
      p2 = pair(p, p);
    }
    const ulonglong2* B = reinterpret_cast<const ulonglong2*>(&sm.bc[0][t][n0]);
    const ulonglong2* C = reinterpret_cast<const ulonglong2*>(&sm.bc[1][t][n0]);
#pragma unroll
    for (int q = 0; q < kStates / 4; ++q) {
      const ulonglong2 bq = B[q];
      const f32x2 a0 = exp2_pair(mul2(A2[2 * q], u2)), a1 = exp2_pair(mul2(A2[2 * q + 1], u2));
      h[2 * q] = fma2(a0, h[2 * q], mul2(g2, bq.x));
      h[2 * q + 1] = fma2(a1, h[2 * q + 1], mul2(g2, bq.y));
      if (CUT && !cleared) {
        const ulonglong2 cq = C[q];
        P[2 * q] = mul2(P[2 * q], a0);
        P[2 * q + 1] = mul2(P[2 * q + 1], a1);
        e[2 * q] = fma2(P[2 * q], mul2(cq.x, p2), e[2 * q]);
        e[2 * q + 1] = fma2(P[2 * q + 1], mul2(cq.y, p2), e[2 * q + 1]);
      }
    }
  };

  fetch(t_begin);
  __syncthreads();
  stage(t_begin);
  __syncthreads();
  for (int t0 = t_begin; t0 < t_end; t0 += L::kTile) {
    fetch(t0 + L::kTile);
    const size_t tile = static_cast<size_t>(b) * sp.tiles + t0 / L::kTile;
    if (live) {
      put(sp.kept + tile * state, h);
      if (n0 == 0) sp.kept_sum[tile * a.D + c] = usum;
    }
    if (blockIdx.x == 0 && tid == 0) sp.kept_clear[tile] = cleared;
    const int nt = min(L::kTile, t_end - t0);
    const unsigned starts = sm.starts[0];
    if (starts == 0 && nt == L::kTile) {
#pragma unroll 4
      for (int t = 0; t < L::kTile; ++t) token(t, false);
    } else {
      for (int t = 0; t < nt; ++t) token(t, (starts >> t) & 1);
    }
    __syncthreads();
    if (t0 + L::kTile < t_end) {
      stage(t0 + L::kTile);
      __syncthreads();
    }
  }
  if (!CUT) return;
  const size_t at = static_cast<size_t>(b) * sp.segments + seg;
  const bool last = seg == sp.segments - 1;
  if (live) {
    if (!last) {
      put(sp.h + (at + 1) * state, h);
      if (n0 == 0) sp.total[at * a.D + c] = usum;
    } else {
      float v[kStates];
#pragma unroll
      for (int i = 0; i < kStates; ++i) v[i] = 0.f;
      if (a.dhT) load8(a.dhT + b * state + own, v);
      f32x2 d[kStates / 2];
#pragma unroll
      for (int i = 0; i < kStates / 2; ++i) {
        d[i] = pair(v[2 * i], v[2 * i + 1]);
        if (!cleared) e[i] = fma2(P[i], d[i], e[i]);
      }
      put(sp.e + at * state, d);
    }
    if (seg > 0) put(sp.e + (at - 1) * state, e);
  }
  if (blockIdx.x == 0 && tid == 0) sp.cleared[at] = cleared;
}

// ------------------------------------------------------------------ gradients

constexpr int kWarps = 4;
constexpr int kBwdThreads = 32 * kWarps;
constexpr int kTile = kSpaceTile;
constexpr int kSub = 4;           // tokens whose decays and states are in registers

template <int N>
struct BwdLayout {
  static constexpr int kStateLanes = N / 4, kChannelLanes = 32 / kStateLanes;
  static constexpr int kWarpChannels = 4 * kChannelLanes, kChannels = kWarps * kWarpChannels;
  static constexpr int kStateMask = (kStateLanes - 1) & 3;       // orders of the channels
  static constexpr int kChannelMask = (kChannelLanes - 1) & 3;   // orders of the states
  static constexpr int kVecs = kTile * kChannels / 8;
  static constexpr int kPer = (kVecs + kBwdThreads - 1) / kBwdThreads;
  static constexpr int kBcVecs = 2 * kTile * N / 8;
  static constexpr int kRow = kChannels / 8;                     // vectors of a token
  static constexpr int kOrder = kTile * N + N;                   // floats of one order of B or C
};

template <int N>
struct __align__(16) BwdShared {
  using L = BwdLayout<N>;
  float u[kTile][L::kChannels], g[kTile][L::kChannels], p[kTile][L::kChannels];
  float q[kTile][L::kChannels], r[kTile][L::kChannels], y[kTile][L::kChannels];
  float b[4][L::kOrder], c[4][L::kOrder];
  float4 h[kTile / kSub][4][kBwdThreads];
  float dbc[kWarps][kTile][2 * N];
  float sums[kBwdThreads][17];        // dskip and ddt_bias of a thread's 8 channels
  float bias[L::kChannels], skip[L::kChannels];
  unsigned starts[4];
};

// v[i] -> v[i ^ mask]
template <typename V>
__device__ __forceinline__ void reorder(V (&v)[4], int mask) {
  if (mask & 1) {
    V s = v[0]; v[0] = v[1]; v[1] = s;
    s = v[2]; v[2] = v[3]; v[3] = s;
  }
  if (mask & 2) {
    V s = v[0]; v[0] = v[2]; v[2] = s;
    s = v[1]; v[1] = v[3]; v[3] = s;
  }
}

__device__ __forceinline__ float pass(float x, int lanes) {
  return __shfl_xor_sync(0xffffffffu, x, lanes);
}

template <typename T, int N, bool Z>
__global__ void __launch_bounds__(kBwdThreads, 2)
    space_bwd_kernel(const SpaceArgs a, const SpaceSplit sp) {
  using L = BwdLayout<N>;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  BwdShared<N>& sm = *reinterpret_cast<BwdShared<N>*>(raw_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane % L::kStateLanes, cl = lane / L::kStateLanes;
  const Channels ch(a, L::kChannels, blockIdx.x);
  const int seg = blockIdx.y, b = blockIdx.z;
  const int t_begin = seg * sp.seg_len, t_end = min(t_begin + sp.seg_len, a.T);
  const long long row0 = static_cast<long long>(b) * a.T;
  const size_t state = static_cast<size_t>(a.D) * N;
  const int n0 = 4 * sl;
  const int cx = sl & L::kStateMask, nx = cl & L::kChannelMask;   // this lane's orders
  const int cbase = warp * L::kWarpChannels + 4 * cl;             // of the CTA's channels
  const float* Border = sm.b[nx];
  const float* Corder = sm.c[nx];

  // [channel i: ch.first + cbase + (i ^ cx)][state j: n0 + (j ^ nx)]
  f32x2 A2[4][2], dA[4][2], E[4][2];
  float hs[4][4];      // the state entering the segment
  const bool from_start = seg == 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = ch.first + cbase + (i ^ cx);
    float A[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) hs[i][j] = 0.f;
    if (d < ch.end) {
      const size_t own = static_cast<size_t>(d) * N + n0;
      const float4 A4 = __ldg(reinterpret_cast<const float4*>(a.A + own));
      A[0] = A4.x * kLog2e; A[1] = A4.y * kLog2e; A[2] = A4.z * kLog2e; A[3] = A4.w * kLog2e;
      if (!from_start) chain_states(a, sp, b, seg, d, n0, A, hs[i]);
      // the gradient entering the segment from behind
      const float* from = nullptr;
      int k = sp.segments - 1;
      if (sp.segments == 1)
        from = a.dhT ? a.dhT + b * state + own : nullptr;
      else {
        if (seg < k) --k;
        from = sp.e + (static_cast<size_t>(b) * sp.segments + k) * state + own;
      }
      if (from) {
        const float4 f = *reinterpret_cast<const float4*>(from);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      }
      for (; k > seg; --k) {     // through segment k
        const size_t at = static_cast<size_t>(b) * sp.segments + k;
        const float u = sp.total[at * a.D + d];
        const bool cleared = sp.cleared[at] != 0;
        const float4 f = *reinterpret_cast<const float4*>(sp.e + (at - 1) * state + own);
        const float add[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = cleared ? add[j] : fmaf(exp2_fast(A[j] * u), v[j], add[j]);
      }
    }
    reorder(A, nx);
    reorder(v, nx);
    reorder(hs[i], nx);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      A2[i][j] = pair(A[2 * j], A[2 * j + 1]);
      E[i][j] = pair(v[2 * j], v[2 * j + 1]);
      dA[i][j] = pair(0.f, 0.f);
    }
  }
  for (int i = tid; i < L::kChannels; i += kBwdThreads) {
    const int d = ch.first + i;
    sm.bias[i] = a.dt_bias && d < ch.end ? a.dt_bias[d] : 0.f;
    sm.skip[i] = a.skip && d < ch.end ? a.skip[d] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sm.sums[tid][i] = 0.f;
  __syncthreads();

  for (int t0 = (t_end - 1) / kTile * kTile; t0 >= t_begin; t0 -= kTile) {
    const int nt = min(kTile, t_end - t0);
    // (u, u x, p) of the tile, B and C in all orders
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kBwdThreads, t = v / L::kRow, d = 8 * (v % L::kRow);
      if (v >= L::kVecs) break;
      float x[8], u[8], p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = u[j] = p[j] = 0.f;
      if (t < nt && ch.first + d < ch.end) {
        const long long row = row0 + t0 + t;
        load8(static_cast<const T*>(a.x) + row * a.xs + ch.first + d, x);
        load8(static_cast<const T*>(a.dt) + row * a.dts + ch.first + d, u);
        load8(static_cast<const T*>(a.dy) + row * a.D + ch.first + d, p);
        float z[8];
        if (Z) load8(static_cast<const T*>(a.z) + row * a.zs + ch.first + d, z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[j] += sm.bias[d + j];
          if (a.softplus) u[j] = softplus(u[j]);
          x[j] *= u[j];
          if (Z) p[j] *= silu(z[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        *reinterpret_cast<float4*>(&sm.u[t][d + 4 * j]) =
            make_float4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
        *reinterpret_cast<float4*>(&sm.g[t][d + 4 * j]) =
            make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
        *reinterpret_cast<float4*>(&sm.p[t][d + 4 * j]) =
            make_float4(p[4 * j], p[4 * j + 1], p[4 * j + 2], p[4 * j + 3]);
      }
    }
    for (int v = tid; v < L::kBcVecs; v += kBwdThreads) {
      const int which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = w / (N / 8), n = 8 * (w % (N / 8));
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.f;
      if (t < nt)
        load8((which ? static_cast<const T*>(a.Cm) + (row0 + t0 + t) * a.cs
                     : static_cast<const T*>(a.Bm) + (row0 + t0 + t) * a.bs) + ch.group * N + n, x);
#pragma unroll
      for (int o = 0; o < 4; ++o)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>((which ? sm.c[o] : sm.b[o]) + t * N + n + 4 * j) =
              make_float4(x[4 * j + (0 ^ o)], x[4 * j + (1 ^ o)], x[4 * j + (2 ^ o)],
                          x[4 * j + (3 ^ o)]);
    }
    {
      const bool mark = a.starts && tid < nt && a.starts[row0 + t0 + tid] != 0;
      const unsigned m = __ballot_sync(0xffffffffu, mark);
      if (tid == 0) sm.starts[0] = m;
    }
    // the tile's first state
    f32x2 h[4][2];
    const size_t tile = static_cast<size_t>(b) * sp.tiles + t0 / kTile;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = ch.first + cbase + (i ^ cx);
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (d < ch.end) {
        const float4 f = *reinterpret_cast<const float4*>(sp.kept + tile * state +
                                                          static_cast<size_t>(d) * N + n0);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        reorder(v, nx);
        if (!from_start && sp.kept_clear[tile] == 0) {
          const float u = sp.kept_sum[tile * a.D + d];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float lo, hi;
            split(A2[i][j], lo, hi);
            v[2 * j] = fmaf(exp2_fast(lo * u), hs[i][2 * j], v[2 * j]);
            v[2 * j + 1] = fmaf(exp2_fast(hi * u), hs[i][2 * j + 1], v[2 * j + 1]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) h[i][j] = pair(v[2 * j], v[2 * j + 1]);
    }
    __syncthreads();
    const unsigned starts = sm.starts[0];

    // forward through the tile, a state kept every kSub tokens
    const int subs = (nt + kSub - 1) / kSub;
    for (int s = 0; s < subs; ++s) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4 f;
        split(h[i][0], f.x, f.y);
        split(h[i][1], f.z, f.w);
        sm.h[s][i][tid] = f;
      }
      if (s + 1 == subs) break;
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        const int t = s * kSub + k;
        if ((starts >> t) & 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i][0] = h[i][1] = pair(0.f, 0.f);
        }
        const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(Border + t * N + n0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = sm.u[t][cbase + (i ^ cx)], g = sm.g[t][cbase + (i ^ cx)];
          const f32x2 u2 = pair(u, u), g2 = pair(g, g);
          h[i][0] = fma2(exp2_pair(mul2(A2[i][0], u2)), h[i][0], mul2(g2, B.x));
          h[i][1] = fma2(exp2_pair(mul2(A2[i][1], u2)), h[i][1], mul2(g2, B.y));
        }
      }
    }
    // and back
    for (int s = subs - 1; s >= 0; --s) {
      f32x2 da[kSub][4][2], ah[kSub][4][2];     // decays, decayed states
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 f = sm.h[s][i][tid];
        h[i][0] = pair(f.x, f.y);
        h[i][1] = pair(f.z, f.w);
      }
      // tokens behind the end have u = u x = p = B = C = 0: they change nothing
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        const int t = s * kSub + k;
        const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(Border + t * N + n0);
        const bool first = (starts >> t) & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float u = sm.u[t][cbase + (i ^ cx)], g = sm.g[t][cbase + (i ^ cx)];
          const f32x2 u2 = pair(u, u), g2 = pair(g, g);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            da[k][i][j] = exp2_pair(mul2(A2[i][j], u2));
            ah[k][i][j] = mul2(da[k][i][j], h[i][j]);
            if (first) ah[k][i][j] = pair(0.f, 0.f);
            h[i][j] = fma2(g2, j ? B.y : B.x, ah[k][i][j]);
          }
        }
      }
#pragma unroll
      for (int k = kSub - 1; k >= 0; --k) {
        const int t = s * kSub + k;
        const ulonglong2 B = *reinterpret_cast<const ulonglong2*>(Border + t * N + n0);
        const ulonglong2 C = *reinterpret_cast<const ulonglong2*>(Corder + t * N + n0);
        f32x2 db[2], dc[2];
        float q[4], r[4], y[4];
        db[0] = db[1] = dc[0] = dc[1] = pair(0.f, 0.f);
        const bool first = (starts >> t) & 1;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = cbase + (i ^ cx);
          const float u = sm.u[t][at], g = sm.g[t][at], p = sm.p[t][at];
          const f32x2 u2 = pair(u, u), g2 = pair(g, g), p2 = pair(p, p);
          f32x2 qq = pair(0.f, 0.f), rr = qq, yy = qq;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const f32x2 Bj = j ? B.y : B.x, Cj = j ? C.y : C.x;
            const f32x2 e = fma2(Cj, p2, E[i][j]);
            const f32x2 ht = fma2(g2, Bj, ah[k][i][j]);
            const f32x2 w = mul2(e, ah[k][i][j]);
            db[j] = fma2(g2, e, db[j]);
            dc[j] = fma2(p2, ht, dc[j]);
            qq = fma2(Bj, e, qq);
            rr = fma2(A2[i][j], w, rr);
            dA[i][j] = fma2(u2, w, dA[i][j]);
            if (Z) yy = fma2(Cj, ht, yy);
            E[i][j] = mul2(da[k][i][j], e);
            if (first) E[i][j] = pair(0.f, 0.f);
          }
          q[i] = sum2(qq);
          r[i] = sum2(rr);
          if (Z) y[i] = sum2(yy);
        }
        // over the state lanes: by halves over the 4 channels, then whole
        auto over_states = [&](float (&v)[4], float* out) {
          v[0] += pass(v[1], 1);
          v[2] += pass(v[3], 1);
          if constexpr (L::kStateLanes >= 4) v[0] += pass(v[2], 2);
          if constexpr (L::kStateLanes >= 8) v[0] += pass(v[0], 4);
          if constexpr (L::kStateLanes >= 16) v[0] += pass(v[0], 8);
          if (sl < 4) {
            out[cbase + cx] = v[0];
            if (L::kStateLanes == 2) out[cbase + (2 ^ cx)] = v[2];
          }
        };
        over_states(q, sm.q[t]);
        over_states(r, sm.r[t]);
        if (Z) over_states(y, sm.y[t]);
        // over the channel lanes
        float vb[4], vc[4];
        split(db[0], vb[0], vb[1]);
        split(db[1], vb[2], vb[3]);
        split(dc[0], vc[0], vc[1]);
        split(dc[1], vc[2], vc[3]);
        constexpr int kStep = L::kStateLanes;     // lanes to the next channel lane
        vb[0] += pass(vb[1], kStep);
        vb[2] += pass(vb[3], kStep);
        vc[0] += pass(vc[1], kStep);
        vc[2] += pass(vc[3], kStep);
        float* out = sm.dbc[warp][t];
        if constexpr (L::kChannelLanes >= 4) {
          vb[0] += pass(vb[2], 2 * kStep);
          vc[0] += pass(vc[2], 2 * kStep);
          if constexpr (L::kChannelLanes >= 8) {
            // one half of the lanes goes on with dB, the other with dC
            const bool up = cl & 4;
            float keep = up ? vc[0] : vb[0];
            keep += pass(up ? vb[0] : vc[0], 4 * kStep);
            if constexpr (L::kChannelLanes >= 16) keep += pass(keep, 8 * kStep);
            if (cl < 8) out[(up ? N : 0) + n0 + nx] = keep;
          } else {
            out[n0 + nx] = vb[0];
            out[N + n0 + nx] = vc[0];
          }
        } else {
          out[n0 + nx] = vb[0];
          out[n0 + (2 ^ nx)] = vb[2];
          out[N + n0 + nx] = vc[0];
          out[N + n0 + (2 ^ nx)] = vc[2];
        }
      }
    }
    __syncthreads();

    // the tile's outputs
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kBwdThreads, t = v / L::kRow, d = 8 * (v % L::kRow);
      if (v >= L::kVecs || t >= nt || ch.first + d >= ch.end) continue;
      const long long row = row0 + t0 + t;
      const size_t out = static_cast<size_t>(row) * a.D + ch.first + d;
      float x[8], raw[8], dy[8], z[8], dx[8], ddt[8], dz[8];
      load8(static_cast<const T*>(a.x) + row * a.xs + ch.first + d, x);
      load8(static_cast<const T*>(a.dt) + row * a.dts + ch.first + d, raw);
      if (Z) {
        load8(static_cast<const T*>(a.dy) + row * a.D + ch.first + d, dy);
        load8(static_cast<const T*>(a.z) + row * a.zs + ch.first + d, z);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float q = sm.q[t][d + j], p = sm.p[t][d + j], sk = sm.skip[d + j];
        dx[j] = sm.u[t][d + j] * q;
        if (a.skip) dx[j] = fmaf(sk, p, dx[j]);
        // A2 is log2(e) A
        ddt[j] = fmaf(x[j], q, sm.r[t][d + j] * (1.f / kLog2e));
        if (a.softplus) ddt[j] *= sigmoid(raw[j] + sm.bias[d + j]);
        if (Z) {
          float y = sm.y[t][d + j];
          if (a.skip) y = fmaf(sk, x[j], y);
          dz[j] = dy[j] * y * silu_slope(z[j]);
        }
        sm.sums[tid][j] = fmaf(p, x[j], sm.sums[tid][j]);
        sm.sums[tid][8 + j] += ddt[j];
      }
      store8(static_cast<T*>(a.dx) + out, dx);
      store8(static_cast<T*>(a.ddt) + out, ddt);
      if (Z) store8(static_cast<T*>(a.dz) + out, dz);
    }
    const int blocks = gridDim.x / a.G, block = blockIdx.x % blocks;
    for (int i = tid; i < nt * 2 * N; i += kBwdThreads) {
      const int t = i / (2 * N), j = i % (2 * N);
      float s = sm.dbc[0][t][j];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s += sm.dbc[w][t][j];
      sp.bc_part[(((static_cast<size_t>(block) * a.B + b) * a.T + t0 + t) * a.G + ch.group) * 2 * N +
                 j] = s;
    }
    __syncthreads();
  }

  const size_t part = static_cast<size_t>(b) * sp.segments + seg;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int d = ch.first + cbase + (i ^ cx);
    if (d >= ch.end) continue;
    const size_t own = static_cast<size_t>(d) * N + n0;
    float v[4];
    split(dA[i][0], v[0], v[1]);
    split(dA[i][1], v[2], v[3]);
    reorder(v, nx);
    *reinterpret_cast<float4*>(sp.dA_part + part * state + own) = make_float4(v[0], v[1], v[2], v[3]);
    if (seg == 0 && a.dh0) {
      split(E[i][0], v[0], v[1]);
      split(E[i][1], v[2], v[3]);
      reorder(v, nx);
      *reinterpret_cast<float4*>(a.dh0 + b * state + own) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
  // dskip and ddt_bias: threads kRow apart have the same channels
  for (int i = tid; i < 2 * L::kChannels; i += kBwdThreads) {
    const int which = i / L::kChannels, d = i % L::kChannels;
    float s = 0.f;
    for (int k = d / 8; k < kBwdThreads; k += L::kRow) s += sm.sums[k][8 * which + d % 8];
    if (ch.first + d < ch.end) sp.d_part[(part * 2 + which) * a.D + ch.first + d] = s;
  }
}

// Adds up the partial sums: dBm and dCm over the CTAs' channels, dA, dskip and ddt_bias over
// batch rows and segments.
template <typename T>
__global__ void __launch_bounds__(256) space_sums_kernel(const SpaceArgs a, const SpaceSplit sp) {
  const long long bc = static_cast<long long>(a.B) * a.T * a.G * 2 * a.N;
  const long long da = static_cast<long long>(a.D) * a.N;
  const int parts = a.B * sp.segments;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < bc + da + 2 * a.D;
       i += static_cast<long long>(gridDim.x) * 256) {
    float s = 0.f;
    if (i < bc) {
#pragma unroll 4
      for (int k = 0; k < sp.blocks; ++k) s += sp.bc_part[k * bc + i];
      const int n = static_cast<int>(i % a.N), which = static_cast<int>(i / a.N % 2);
      const long long at = i / (2 * a.N) * a.N + n;
      static_cast<T*>(which ? a.dCm : a.dBm)[at] = static_cast<T>(s);
    } else if (i < bc + da) {
#pragma unroll 4
      for (int k = 0; k < parts; ++k) s += sp.dA_part[k * da + i - bc];
      a.dA[i - bc] = s;
    } else {
      const long long j = i - bc - da;
#pragma unroll 4
      for (int k = 0; k < parts; ++k) s += sp.d_part[k * 2 * a.D + j];
      if (j < a.D) {
        if (a.skip) a.dskip[j] = s;
      } else if (a.dt_bias) {
        a.ddt_bias[j - a.D] = s;
      }
    }
  }
}

template <class F>
cudaError_t by_states(int N, bool f32, F f) {
  using std::integral_constant;
  auto typed = [&](auto n) { return f32 ? f(float{}, n) : f(__nv_bfloat16{}, n); };
  if (N == 8) return typed(integral_constant<int, 8>{});
  if (N == 16) return typed(integral_constant<int, 16>{});
  if (N == 32) return typed(integral_constant<int, 32>{});
  return typed(integral_constant<int, 64>{});
}

int blocks_of(const SpaceArgs& a, int channels) {
  const int each = a.D / a.G;
  return (each + channels - 1) / channels;
}

}  // namespace

int space_channels(int N, bool backward) {
  return backward ? kWarps * 4 * 32 / (N / 4) : kThreads / (N / kStates);
}

cudaError_t launch_space_bwd_states(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                                    cudaStream_t stream) {
  return by_states(a.N, f32, [&](auto t, auto n) {
    constexpr int kBytes = static_cast<int>(sizeof(PreShared<n>));
    auto* kern = sp.segments > 1 ? space_bwd_states_kernel<decltype(t), n, true>
                                 : space_bwd_states_kernel<decltype(t), n, false>;
    const cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (err != cudaSuccess) return err;
    kern<<<dim3(a.G * blocks_of(a, PreLayout<n>::kChannels), sp.segments, a.B), kThreads, kBytes,
           stream>>>(a, sp);
    return cudaGetLastError();
  });
}

cudaError_t launch_space_bwd(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                             cudaStream_t stream) {
  const cudaError_t err = by_states(a.N, f32, [&](auto t, auto n) {
    constexpr int kBytes = static_cast<int>(sizeof(BwdShared<n>));
    auto* kern = a.z ? space_bwd_kernel<decltype(t), n, true> : space_bwd_kernel<decltype(t), n, false>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    kern<<<dim3(a.G * blocks_of(a, BwdLayout<n>::kChannels), sp.segments, a.B), kBwdThreads, kBytes,
           stream>>>(a, sp);
    return cudaGetLastError();
  });
  if (err != cudaSuccess) return err;
  const long long n = static_cast<long long>(a.B) * a.T * a.G * 2 * a.N +
                      static_cast<long long>(a.D) * (a.N + 2);
  const long long want = (n + 255) / 256;
  const unsigned grid = static_cast<unsigned>(want < 152 * 32 ? want : 152 * 32);
  if (f32)
    space_sums_kernel<float><<<grid, 256, 0, stream>>>(a, sp);
  else
    space_sums_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, sp);
  return cudaGetLastError();
}

}  // namespace gdr
