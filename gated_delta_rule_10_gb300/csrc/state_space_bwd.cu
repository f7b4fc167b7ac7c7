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
// Three exponentials and about 22 multiply-adds for each (token, channel, state) in all. The
// second launch is 73% of the time (4 x 4096 x 2048 channels x 16 bf16: 756 us in all): two
// warps a scheduler, which 255 registers a thread and 111 KB of shared memory a CTA leave,
// issue 51% of the time. With half the states a thread (three CTAs an SM) it issues 58% of the
// time but 30% more, and takes as long; so does half the tokens in registers. Tiles without a
// document's start take a walk without branches (851 -> 831 us), whole tiles are staged and
// finished without them (804 -> 770).
//
// A thread has 4 states of 4 channels (pairs of channels share an instruction), so that the
// sums over channels (dB, dC) and those over states (q, sum A w, C h) each start inside a
// thread. What is left goes over lanes by halves: a lane passes on half of its sums and keeps
// the other half. Which one is by lane, so a lane's registers hold its states in the order
// n ^ lane (pairs of channels alike), and no register has to be selected; B and C are in
// shared memory in all four orders.
#include <type_traits>

#include "state_space.cuh"

namespace gdr {
namespace {

// ------------------------------------------------------------------ states

constexpr int kThreads = 128;
constexpr int kStates = 8;        // states of a thread, of each of its channels
constexpr int kOwn = 2;           // channels of a thread

template <int N>
struct PreLayout {
  static constexpr int kLanes = N / kStates;
  static constexpr int kChannels = kOwn * kThreads / kLanes;
  static constexpr int kTile = N == 8 ? 8 : kSpaceTile;      // tokens staged together
  static constexpr int kVecs = kTile * kChannels / 8;
  static constexpr int kPer = (kVecs + kThreads - 1) / kThreads;
  static constexpr int kBcVecs = 2 * kTile * N / 8;
  static constexpr int kBcPer = (kBcVecs + kThreads - 1) / kThreads;
};

template <typename T, int N>
struct __align__(16) PreShared {
  using L = PreLayout<N>;
  float u[L::kTile][L::kChannels], g[L::kTile][L::kChannels], p[L::kTile][L::kChannels];
  float bc[2][L::kTile][N];
  T x[L::kTile][L::kChannels], dt[L::kTile][L::kChannels];
  T z[L::kTile][L::kChannels], dy[L::kTile][L::kChannels];
  T raw_bc[2][L::kTile][N];
  float bias[L::kChannels];
  unsigned starts[4];
};

// CUT: there are several segments, which need the gradients that they pass back.
template <typename T, int N, bool CUT>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? (CUT ? 4 : 5) : 1)
    space_bwd_states_kernel(const SpaceArgs a, const SpaceSplit sp) {
  using L = PreLayout<N>;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  PreShared<T, N>& sm = *reinterpret_cast<PreShared<T, N>*>(raw_smem);
  const int tid = threadIdx.x;
  const Channels ch(a, L::kChannels, blockIdx.x);
  const int seg = blockIdx.y, b = blockIdx.z;
  const int t_begin = seg * sp.seg_len, t_end = min(t_begin + sp.seg_len, a.T);
  const long long row0 = static_cast<long long>(b) * a.T;
  const int ci = kOwn * (tid / L::kLanes), c = ch.first + ci, n0 = (tid % L::kLanes) * kStates;
  const bool live = c < ch.end;      // channels come in eights
  const size_t state = static_cast<size_t>(a.D) * N;
  f32x2 A2[kOwn][kStates / 2], h[kOwn][kStates / 2], P[kOwn][kStates / 2], e[kOwn][kStates / 2];
  f32x2 usum = 0;                    // of the two channels
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const size_t own = static_cast<size_t>(c + o) * N + n0;
    float A[kStates], v[kStates];
#pragma unroll
    for (int i = 0; i < kStates; ++i) A[i] = v[i] = 0.f;
    if (live) {
      load8(a.A + own, A);
      if (seg == 0 && a.h0) load8(a.h0 + b * state + own, v);
    }
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) {
      A2[o][i] = pair(A[2 * i] * kLog2e, A[2 * i + 1] * kLog2e);
      h[o][i] = pair(v[2 * i], v[2 * i + 1]);
      P[o][i] = both(1.f);
      e[o][i] = 0;
    }
  }
  for (int i = tid; i < L::kChannels; i += kThreads)
    sm.bias[i] = a.dt_bias && ch.first + i < ch.end ? a.dt_bias[ch.first + i] : 0.f;

  bool mark = false;
  constexpr int kBc = CUT ? L::kBcVecs : L::kBcVecs / 2;
  // copies a tile's inputs
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kThreads, t = v / (L::kChannels / 8), d = 8 * (v % (L::kChannels / 8));
      if (v < L::kVecs && t0 + t < t_end && ch.first + d < ch.end) {
        const long long row = row0 + t0 + t;
        copy8(&sm.x[t][d], static_cast<const T*>(a.x) + row * a.xs + ch.first + d);
        copy8(&sm.dt[t][d], static_cast<const T*>(a.dt) + row * a.dts + ch.first + d);
        if (CUT) {
          copy8(&sm.dy[t][d], static_cast<const T*>(a.dy) + row * a.D + ch.first + d);
          if (a.z) copy8(&sm.z[t][d], static_cast<const T*>(a.z) + row * a.zs + ch.first + d);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = w / (N / 8), n = 8 * (w % (N / 8));
      if (v < kBc && t0 + t < t_end)
        copy8(&sm.raw_bc[which][t][n],
              (which ? static_cast<const T*>(a.Cm) + (row0 + t0 + t) * a.cs
                     : static_cast<const T*>(a.Bm) + (row0 + t0 + t) * a.bs) +
                  ch.group * N + n);
    }
    mark = a.starts && tid < L::kTile && t0 + tid < t_end && a.starts[row0 + t0 + tid] != 0;
  };
  // what this thread has copied, as the walk reads it; PLAIN: nothing of the tile is missing,
  // u is a softplus and there is a gate, so that no branch parts the vectors' long chains
  const bool full = ch.first + L::kChannels <= ch.end;
  auto stage = [&](int t0) {
    copies_done();
    auto steps = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int v = tid + i * kThreads, t = v / (L::kChannels / 8), d = 8 * (v % (L::kChannels / 8));
        if (v >= L::kVecs) break;
        f32x2 x[4], u[4], p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = u[j] = p[j] = 0;
        if (PLAIN || (t0 + t < t_end && ch.first + d < ch.end)) {
          f32x2 bias[4], z[4];
          read8(&sm.x[t][d], x);
          read8(&sm.dt[t][d], u);
          read8(&sm.bias[d], bias);
          if (CUT) read8(&sm.dy[t][d], p);
          if (CUT && (PLAIN || a.z)) read8(&sm.z[t][d], z);
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = add2(u[j], bias[j]);
          if (PLAIN || a.softplus)
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = softplus2(u[j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = mul2(u[j], x[j]);
          if (CUT && (PLAIN || a.z))
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = mul2(p[j], mul2(z[j], sigmoid2(z[j])));
        }
        write8(&sm.u[t][d], u);
        write8(&sm.g[t][d], x);
        if (CUT) write8(&sm.p[t][d], p);
      }
    };
    if (full && a.softplus && (!CUT || a.z) && t0 + L::kTile <= t_end)
      steps(std::true_type{});
    else
      steps(std::false_type{});
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = w / (N / 8), n = 8 * (w % (N / 8));
      if (v >= kBc) break;
      f32x2 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = 0;
      if (t0 + t < t_end) read8(&sm.raw_bc[which][t][n], x);
      write8(&sm.bc[which][t][n], x);
    }
    const unsigned m = __ballot_sync(0xffffffffu, mark);
    if (tid == 0) sm.starts[0] = m;
  };
  auto put = [&](float* out, const f32x2 (&v)[kOwn][kStates / 2]) {
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      ulonglong2* p = reinterpret_cast<ulonglong2*>(out + static_cast<size_t>(c + o) * N + n0);
      p[0] = make_ulonglong2(v[o][0], v[o][1]);
      p[1] = make_ulonglong2(v[o][2], v[o][3]);
    }
  };

  bool cleared = false;     // a document starts in what has been walked of the segment
  // one token, which may be a document's first; `back`: with what it passes back (nothing
  // from a document that starts in the segment)
  auto token = [&](int t, bool first, bool back) {
    const float2 u = *reinterpret_cast<const float2*>(&sm.u[t][ci]);
    const float2 g = *reinterpret_cast<const float2*>(&sm.g[t][ci]);
    if (first) {
      cleared = true;
      back = false;
#pragma unroll
      for (int o = 0; o < kOwn; ++o)
#pragma unroll
        for (int i = 0; i < kStates / 2; ++i) h[o][i] = P[o][i] = 0;
    }
    usum = add2(usum, pair(u.x, u.y));
    const f32x2 u2[kOwn] = {both(u.x), both(u.y)}, g2[kOwn] = {both(g.x), both(g.y)};
    f32x2 p2[kOwn];
    if (back) {
      const float2 p = *reinterpret_cast<const float2*>(&sm.p[t][ci]);
      p2[0] = both(p.x);
      p2[1] = both(p.y);
    }
    const ulonglong2* B = reinterpret_cast<const ulonglong2*>(&sm.bc[0][t][n0]);
    const ulonglong2* C = reinterpret_cast<const ulonglong2*>(&sm.bc[1][t][n0]);
#pragma unroll
    for (int q = 0; q < kStates / 4; ++q) {
      const ulonglong2 bq = B[q];
      ulonglong2 cq;
      if (back) cq = C[q];
#pragma unroll
      for (int o = 0; o < kOwn; ++o)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int i = 2 * q + j;
          const f32x2 d = decay2(A2[o][i], u2[o]);
          h[o][i] = fma2(g2[o], j ? bq.y : bq.x, mul2(d, h[o][i]));
          if (back) {
            P[o][i] = mul2(d, P[o][i]);
            e[o][i] = fma2(P[o][i], mul2(j ? cq.y : cq.x, p2[o]), e[o][i]);
          }
        }
    }
  };

  fetch(t_begin);
  __syncthreads();
  stage(t_begin);
  __syncthreads();
  for (int t0 = t_begin; t0 < t_end; t0 += L::kTile) {
    fetch(t0 + L::kTile);
    if (t0 % kSpaceTile == 0) {
      const size_t tile = static_cast<size_t>(b) * sp.tiles + t0 / kSpaceTile;
      if (live) {
        put(sp.kept + tile * state, h);
        if (n0 == 0) *reinterpret_cast<f32x2*>(sp.kept_sum + tile * a.D + c) = usum;
      }
      if (blockIdx.x == 0 && tid == 0) sp.kept_clear[tile] = cleared;
    }
    const int nt = min(L::kTile, t_end - t0);
    const unsigned starts = sm.starts[0];
    if (starts == 0 && nt == L::kTile) {
      if (CUT && !cleared) {
#pragma unroll
        for (int t = 0; t < L::kTile; ++t) token(t, false, true);
      } else {
#pragma unroll
        for (int t = 0; t < L::kTile; ++t) token(t, false, false);
      }
    } else {
      for (int t = 0; t < nt; ++t) token(t, (starts >> t) & 1, CUT && !cleared);
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
      if (n0 == 0) *reinterpret_cast<f32x2*>(sp.total + at * a.D + c) = usum;
    } else {
      f32x2 d[kOwn][kStates / 2];
#pragma unroll
      for (int o = 0; o < kOwn; ++o) {
        float v[kStates];
#pragma unroll
        for (int i = 0; i < kStates; ++i) v[i] = 0.f;
        if (a.dhT) load8(a.dhT + b * state + static_cast<size_t>(c + o) * N + n0, v);
#pragma unroll
        for (int i = 0; i < kStates / 2; ++i) {
          d[o][i] = pair(v[2 * i], v[2 * i + 1]);
          if (!cleared) e[o][i] = fma2(P[o][i], d[o][i], e[o][i]);
        }
      }
      put(sp.e + at * state, d);
    }
    if (seg > 0) put(sp.e + (at - 1) * state, e);
  }
  if (blockIdx.x == 0 && tid == 0) sp.cleared[at] = cleared;
}

// ------------------------------------------------------------------ gradients

constexpr int kTile = kSpaceTile;
constexpr int kSub = 4;           // tokens whose decays and states are in registers

// Warps of a CTA. Of shared memory two CTAs have room on an SM, which are 8 warps, or 4 with 8
// states (86 KB each); of fp32 one with 16 states (147 KB), and with 8 three of one warp.
constexpr int bwd_warps(int N, bool f32) {
  if (N == 8) return f32 ? 1 : 2;      // (fp32: 641 us for 4 x 4096 x 1024 with two, 524)
  return 4;
}

template <int N, bool F32>
struct BwdLayout {
  static constexpr int kWarps = bwd_warps(N, F32);
  static constexpr int kBwdThreads = 32 * kWarps;
  static constexpr int kStateLanes = N / 4, kChannelLanes = 32 / kStateLanes;
  static constexpr int kWarpChannels = 4 * kChannelLanes, kChannels = kWarps * kWarpChannels;
  static constexpr int kOrders = kChannelLanes < 4 ? kChannelLanes : 4;   // of the states
  static constexpr int kVecs = kTile * kChannels / 8;
  static constexpr int kPer = (kVecs + kBwdThreads - 1) / kBwdThreads;
  static constexpr int kBcVecs = 2 * kTile * N / 8;
  static constexpr int kBcPer = (kBcVecs + kBwdThreads - 1) / kBwdThreads;
  static constexpr int kRow = kChannels / 8;                     // vectors of a token
  static constexpr int kOrder = kTile * N + N;                   // floats of one order of B or C
  static constexpr int kSums = (kChannels + kBwdThreads - 1) / kBwdThreads;
};

template <typename T, int N, bool Z>
struct __align__(16) BwdShared {
  using L = BwdLayout<N, sizeof(T) == 4>;
  static constexpr int kBwdThreads = L::kBwdThreads;
  // u; u x, then q; p, then C h
  float u[kTile][L::kChannels], g[kTile][L::kChannels], p[kTile][L::kChannels];
  float b[L::kOrders][L::kOrder], c[L::kOrders][L::kOrder];
  // States kept every kSub tokens, a thread's in its own places. Once a warp has taken those of
  // kSub tokens back into registers, its places there (512 bytes for each of the tokens) hold
  // the tokens' sums: 2 N of dB and dC, then, where there is room, sum A w (then ddt) of the
  // warp's channels.
  ulonglong2 h[kTile / kSub][kSub][kBwdThreads];
  float r_apart[N == 64 ? kTile : 1][L::kChannels];
  float px[kBwdThreads][8];           // dskip of a thread's 8 channels
  // copies: two tiles' inputs, and the next tile's first states
  float4 kept[4][kBwdThreads];
  T x[2][kTile][L::kChannels], dt[2][kTile][L::kChannels], dy[2][kTile][L::kChannels];
  T z[2][Z ? kTile : 1][L::kChannels];
  T bc[2][kTile][N];
  float bias[L::kChannels], skip[L::kChannels];
  unsigned starts[4];

  __device__ __forceinline__ float* dbc(int warp, int t) {
    return reinterpret_cast<float*>(&h[t / kSub][t % kSub][32 * warp]);
  }
  __device__ __forceinline__ float* r(int t, int c) {
    if (N == 64) return &r_apart[t][c];
    return dbc(c / L::kWarpChannels, t) + 2 * N + c % L::kWarpChannels;
  }
};

// v[i] -> v[i ^ mask]
__device__ __forceinline__ void reorder(float (&v)[4], int mask) {
  if (mask & 1) {
    float s = v[0]; v[0] = v[1]; v[1] = s;
    s = v[2]; v[2] = v[3]; v[3] = s;
  }
  if (mask & 2) {
    float s = v[0]; v[0] = v[2]; v[2] = s;
    s = v[1]; v[1] = v[3]; v[3] = s;
  }
}
// A thread's states: pairs of channels, in its order of the states.
using Items = f32x2[2][4];
__device__ __forceinline__ void to_items(const float4 (&in)[4], int order, Items& out) {
  float v[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i][0] = in[i].x; v[i][1] = in[i].y; v[i][2] = in[i].z; v[i][3] = in[i].w;
    reorder(v[i], order);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) out[p][j] = pair(v[2 * p][j], v[2 * p + 1][j]);
}
__device__ __forceinline__ void from_items(const Items& in, int order, float4 (&out)[4]) {
  float v[4][4];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) split(in[p][j], v[2 * p][j], v[2 * p + 1][j]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    reorder(v[i], order);
    out[i] = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
  }
}

__device__ __forceinline__ float pass(float x, int lanes) {
  return __shfl_xor_sync(0xffffffffu, x, lanes);
}
template <typename T, int N, bool Z>
__global__ void __launch_bounds__(BwdLayout<N, sizeof(T) == 4>::kBwdThreads, 2)
    space_bwd_kernel(const SpaceArgs a, const SpaceSplit sp) {
  using L = BwdLayout<N, sizeof(T) == 4>;
  constexpr int kWarps = L::kWarps, kBwdThreads = L::kBwdThreads;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  BwdShared<T, N, Z>& sm = *reinterpret_cast<BwdShared<T, N, Z>*>(raw_smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int sl = lane % L::kStateLanes, cl = lane / L::kStateLanes;
  const Channels ch(a, L::kChannels, blockIdx.x);
  const int seg = blockIdx.y, b = blockIdx.z;
  const int t_begin = seg * sp.seg_len, t_end = min(t_begin + sp.seg_len, a.T);
  const long long row0 = static_cast<long long>(b) * a.T;
  const size_t state = static_cast<size_t>(a.D) * N;
  const int n0 = 4 * sl, nx = cl & (L::kOrders - 1);     // states n0 + (j ^ nx)
  const int swap = sl & 1;                               // channels 2 (p ^ swap) + 0, 1
  const int cbase = warp * L::kWarpChannels + 4 * cl;    // of the CTA's channels
  const int c0 = cbase + 2 * swap, c1 = cbase + 2 * (swap ^ 1);
  const bool live = ch.first + cbase < ch.end;           // channels come in eights
  const float* Border = sm.b[nx];
  const float* Corder = sm.c[nx];
  // place of channel i (of four) in a [D, N] array
  auto place = [&](int i) {
    return static_cast<size_t>(ch.first + (i < 2 ? c0 : c1) + (i & 1)) * N + n0;
  };
  auto load_items = [&](const float* from, Items& out) {
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = live && from ? *reinterpret_cast<const float4*>(from + place(i))
                          : make_float4(0.f, 0.f, 0.f, 0.f);
    to_items(v, nx, out);
  };

  Items A2, dA, E, hs;       // hs: the state entering the segment
  const bool from_start = seg == 0;
  load_items(a.A, A2);
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      A2[p][j] = mul2(A2[p][j], both(kLog2e));
      dA[p][j] = 0;
    }
  const size_t at = static_cast<size_t>(b) * sp.segments + seg;
  load_items(from_start ? nullptr : sp.h + at * state, hs);
  // the gradient entering the segment from behind
  load_items(sp.segments > 1 ? sp.e + at * state : a.dhT ? a.dhT + b * state : nullptr, E);
  for (int i = tid; i < L::kChannels; i += kBwdThreads) {
    const int d = ch.first + i;
    sm.bias[i] = a.dt_bias && d < ch.end ? a.dt_bias[d] : 0.f;
    sm.skip[i] = a.skip && d < ch.end ? a.skip[d] : 0.f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sm.px[tid][i] = 0.f;
  float dbias[L::kSums];
#pragma unroll
  for (int i = 0; i < L::kSums; ++i) dbias[i] = 0.f;

  bool mark = false;
  float ksum[4] = {0.f, 0.f, 0.f, 0.f};      // sums of u up to the tile, of this thread's channels
  bool kclear = false;
  // copies a tile's inputs and the state entering it
  auto fetch = [&](int t0, int buf) {
    const int nt = min(kTile, t_end - t0);
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kBwdThreads, t = v / L::kRow, d = 8 * (v % L::kRow);
      if (v < L::kVecs && t < nt && ch.first + d < ch.end) {
        const long long row = row0 + t0 + t;
        copy8(&sm.x[buf][t][d], static_cast<const T*>(a.x) + row * a.xs + ch.first + d);
        copy8(&sm.dt[buf][t][d], static_cast<const T*>(a.dt) + row * a.dts + ch.first + d);
        copy8(&sm.dy[buf][t][d], static_cast<const T*>(a.dy) + row * a.D + ch.first + d);
        if (Z) copy8(&sm.z[buf][Z ? t : 0][d], static_cast<const T*>(a.z) + row * a.zs + ch.first + d);
      }
    }
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kBwdThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = w / (N / 8), n = 8 * (w % (N / 8));
      if (v < L::kBcVecs && t < nt)
        copy8(&sm.bc[which][t][n],
              (which ? static_cast<const T*>(a.Cm) + (row0 + t0 + t) * a.cs
                     : static_cast<const T*>(a.Bm) + (row0 + t0 + t) * a.bs) +
                  ch.group * N + n);
    }
    const size_t tile = static_cast<size_t>(b) * sp.tiles + t0 / kTile;
    if (live) {
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16(&sm.kept[i][tid], sp.kept + tile * state + place(i));
      if (!from_start) {
        const float2 s0 = *reinterpret_cast<const float2*>(sp.kept_sum + tile * a.D + ch.first + c0);
        const float2 s1 = *reinterpret_cast<const float2*>(sp.kept_sum + tile * a.D + ch.first + c1);
        ksum[0] = s0.x; ksum[1] = s0.y; ksum[2] = s1.x; ksum[3] = s1.y;
      }
    }
    kclear = sp.kept_clear[tile] != 0;
    mark = a.starts && tid < nt && a.starts[row0 + t0 + tid] != 0;
  };

  const int t_last = (t_end - 1) / kTile * kTile;
  fetch(t_last, 0);
  __syncthreads();
  const bool full = ch.first + L::kChannels <= ch.end;
  int buf = 0;
  for (int t0 = t_last; t0 >= t_begin; t0 -= kTile, buf ^= 1) {
    const int nt = min(kTile, t_end - t0);
    copies_done();
    // u, u x and p of what this thread has copied; PLAIN: as above
    const bool plain = full && nt == kTile && a.softplus && a.skip;
    auto steps = [&](auto all) {
      constexpr bool PLAIN = decltype(all)::value;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int v = tid + i * kBwdThreads, t = v / L::kRow, d = 8 * (v % L::kRow);
        if (v >= L::kVecs) break;
        f32x2 x[4], u[4], p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = u[j] = p[j] = 0;
        if (PLAIN || (t < nt && ch.first + d < ch.end)) {
          f32x2 bias[4], z[4];
          read8(&sm.x[buf][t][d], x);
          read8(&sm.dt[buf][t][d], u);
          read8(&sm.dy[buf][t][d], p);
          if (Z) read8(&sm.z[buf][Z ? t : 0][d], z);
          read8(&sm.bias[d], bias);
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = add2(u[j], bias[j]);
          if (PLAIN || a.softplus)
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = softplus2(u[j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[j] = mul2(u[j], x[j]);
            if (Z) p[j] = mul2(p[j], mul2(z[j], sigmoid2(z[j])));
          }
        }
        write8(&sm.u[t][d], u);
        write8(&sm.g[t][d], x);
        write8(&sm.p[t][d], p);
      }
    };
    if (plain)
      steps(std::true_type{});
    else
      steps(std::false_type{});
    // B and C in all orders
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kBwdThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = w / (N / 8), n = 8 * (w % (N / 8));
      if (v >= L::kBcVecs) break;
      f32x2 y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = 0;
      if (t < nt) read8(&sm.bc[which][t][n], y);
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(y[j], x[2 * j], x[2 * j + 1]);
#pragma unroll
      for (int o = 0; o < L::kOrders; ++o)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<float4*>((which ? sm.c[o] : sm.b[o]) + t * N + n + 4 * j) =
              make_float4(x[4 * j + (0 ^ o)], x[4 * j + (1 ^ o)], x[4 * j + (2 ^ o)],
                          x[4 * j + (3 ^ o)]);
    }
    {
      const unsigned m = __ballot_sync(0xffffffffu, mark);
      if (tid == 0) sm.starts[0] = m;
    }
    // the tile's first state: the segment's own, and what is left of the one that enters it
    Items h;
    {
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = live ? sm.kept[i][tid] : make_float4(0.f, 0.f, 0.f, 0.f);
      to_items(v, nx, h);
      if (!from_start && !kclear) {
        const f32x2 k2[2] = {pair(ksum[0], ksum[1]), pair(ksum[2], ksum[3])};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[p][j] = fma2(exp2_pair(mul2(A2[p][j], k2[p])), hs[p][j], h[p][j]);
      }
    }
    __syncthreads();
    if (t0 > t_begin) fetch(t0 - kTile, buf ^ 1);
    const unsigned starts = sm.starts[0];

    // forward through the tile, a state kept every kSub tokens; MARKED: documents may start in
    // the tile (else no branch parts the tokens)
    const int subs = (nt + kSub - 1) / kSub;
    auto forth = [&](int s, auto marked) {
      constexpr bool MARKED = decltype(marked)::value;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          sm.h[s][2 * p + j][tid] = make_ulonglong2(h[p][2 * j], h[p][2 * j + 1]);
      if (s + 1 == subs) return;
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        const int t = s * kSub + k;
        const float4 B = *reinterpret_cast<const float4*>(Border + t * N + n0);
        const f32x2 b2[4] = {both(B.x), both(B.y), both(B.z), both(B.w)};
        const f32x2 u[2] = {*reinterpret_cast<const f32x2*>(&sm.u[t][c0]),
                            *reinterpret_cast<const f32x2*>(&sm.u[t][c1])};
        const f32x2 g[2] = {*reinterpret_cast<const f32x2*>(&sm.g[t][c0]),
                            *reinterpret_cast<const f32x2*>(&sm.g[t][c1])};
        if (MARKED && ((starts >> t) & 1)) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) h[p][j] = 0;
        }
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            h[p][j] = fma2(g[p], b2[j], mul2(decay2(A2[p][j], u[p]), h[p][j]));
      }
    };
    if (starts == 0)
      for (int s = 0; s < subs; ++s) forth(s, std::false_type{});
    else
      for (int s = 0; s < subs; ++s) forth(s, std::true_type{});
    // a token's sums over lanes: q, sum A w and C h over a channel's states, dB and dC over channels
    struct Sums {
      f32x2 q[2], r[2], y[2];
      float b[4], c[4];
    };
    auto over_lanes = [&](int t, Sums& v) {
      // over the state lanes: by halves over the 4 channels, then whole
      auto over_states = [&](const f32x2 (&x)[2], float* out) {      // out: of channel cbase
        float lo, hi, lo1, hi1;
        split(x[0], lo, hi);
        split(x[1], lo1, hi1);
        lo += pass(lo1, 1);
        hi += pass(hi1, 1);
        if constexpr (L::kStateLanes == 2) {
          *reinterpret_cast<float2*>(out + 2 * swap) = make_float2(lo, hi);
        } else {
          const bool up = sl & 2;
          float keep = up ? hi : lo;
          keep += pass(up ? lo : hi, 2);
          if constexpr (L::kStateLanes >= 8) keep += pass(keep, 4);
          if constexpr (L::kStateLanes >= 16) keep += pass(keep, 8);
          if (sl < 4) out[2 * swap + up] = keep;
        }
      };
      over_states(v.q, &sm.g[t][cbase]);
      over_states(v.r, sm.r(t, cbase));
      if (Z) over_states(v.y, &sm.p[t][cbase]);
      // over the channel lanes
      constexpr int kStep = L::kStateLanes;     // lanes to the next channel lane
      v.b[0] += pass(v.b[1], kStep);
      v.b[2] += pass(v.b[3], kStep);
      v.c[0] += pass(v.c[1], kStep);
      v.c[2] += pass(v.c[3], kStep);
      float* out = sm.dbc(warp, t);
      if constexpr (L::kChannelLanes >= 4) {
        v.b[0] += pass(v.b[2], 2 * kStep);
        v.c[0] += pass(v.c[2], 2 * kStep);
        if constexpr (L::kChannelLanes >= 8) {
          // one half of the lanes goes on with dB, the other with dC
          const bool up = cl & 4;
          float keep = up ? v.c[0] : v.b[0];
          keep += pass(up ? v.b[0] : v.c[0], 4 * kStep);
          if constexpr (L::kChannelLanes >= 16) keep += pass(keep, 8 * kStep);
          if (cl < 8) out[(up ? N : 0) + n0 + nx] = keep;
        } else {
          out[n0 + nx] = v.b[0];
          out[N + n0 + nx] = v.c[0];
        }
      } else {
        out[n0 + nx] = v.b[0];
        out[n0 + (2 ^ nx)] = v.b[2];
        out[N + n0 + nx] = v.c[0];
        out[N + n0 + (2 ^ nx)] = v.c[2];
      }
    };
    // and back
    auto back = [&](int s, auto marked) {
      constexpr bool MARKED = decltype(marked)::value;
      Items da[kSub], ah[kSub];     // decays, decayed states
      Sums sums[2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const ulonglong2 v = sm.h[s][2 * p + j][tid];
          h[p][2 * j] = v.x;
          h[p][2 * j + 1] = v.y;
        }
      // (tokens behind the end have u = u x = p = B = C = 0: they change nothing)
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        const int t = s * kSub + k;
        const float4 B = *reinterpret_cast<const float4*>(Border + t * N + n0);
        const f32x2 b2[4] = {both(B.x), both(B.y), both(B.z), both(B.w)};
        const f32x2 u[2] = {*reinterpret_cast<const f32x2*>(&sm.u[t][c0]),
                            *reinterpret_cast<const f32x2*>(&sm.u[t][c1])};
        const f32x2 g[2] = {*reinterpret_cast<const f32x2*>(&sm.g[t][c0]),
                            *reinterpret_cast<const f32x2*>(&sm.g[t][c1])};
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            da[k][p][j] = decay2(A2[p][j], u[p]);
            ah[k][p][j] = mul2(da[k][p][j], h[p][j]);
            h[p][j] = fma2(g[p], b2[j], ah[k][p][j]);
          }
        if (MARKED && ((starts >> t) & 1)) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              ah[k][p][j] = 0;
              h[p][j] = mul2(g[p], b2[j]);
            }
        }
      }
#pragma unroll
      for (int k = kSub - 1; k >= 0; --k) {
        const int t = s * kSub + k;
        const float4 B = *reinterpret_cast<const float4*>(Border + t * N + n0);
        const float4 C = *reinterpret_cast<const float4*>(Corder + t * N + n0);
        const f32x2 b2[4] = {both(B.x), both(B.y), both(B.z), both(B.w)};
        const f32x2 cc[4] = {both(C.x), both(C.y), both(C.z), both(C.w)};
        f32x2 db[4], dc[4];
        f32x2 (&q)[2] = sums[k & 1].q, (&r)[2] = sums[k & 1].r, (&y)[2] = sums[k & 1].y;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int c = p ? c1 : c0;
          const f32x2 u = *reinterpret_cast<const f32x2*>(&sm.u[t][c]);
          const f32x2 g = *reinterpret_cast<const f32x2*>(&sm.g[t][c]);
          const f32x2 pp = *reinterpret_cast<const f32x2*>(&sm.p[t][c]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x2 ahk = ah[k][p][j];
            const f32x2 e = fma2(cc[j], pp, E[p][j]);
            const f32x2 ht = fma2(g, b2[j], ahk);
            const f32x2 w = mul2(e, ahk);
            db[j] = p ? fma2(g, e, db[j]) : mul2(g, e);
            dc[j] = p ? fma2(pp, ht, dc[j]) : mul2(pp, ht);
            q[p] = j ? fma2(b2[j], e, q[p]) : mul2(b2[j], e);
            r[p] = j ? fma2(A2[p][j], w, r[p]) : mul2(A2[p][j], w);
            if (Z) y[p] = j ? fma2(cc[j], ht, y[p]) : mul2(cc[j], ht);
            dA[p][j] = fma2(u, w, dA[p][j]);
            E[p][j] = mul2(da[k][p][j], e);
          }
        }
        if (MARKED && ((starts >> t) & 1)) {
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int j = 0; j < 4; ++j) E[p][j] = 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sums[k & 1].b[j] = sum2(db[j]);
          sums[k & 1].c[j] = sum2(dc[j]);
        }
        // a token's sums go over the lanes behind the next one's loads, which would else wait
        // for them to be written (8 states 2%, 32 and 64 states and fp32 1% faster)
        if (k < kSub - 1) over_lanes(t + 1, sums[(k + 1) & 1]);
      }
      over_lanes(s * kSub, sums[0]);
    };
    if (starts == 0)
      for (int s = subs - 1; s >= 0; --s) back(s, std::false_type{});
    else
      for (int s = subs - 1; s >= 0; --s) back(s, std::true_type{});

    // the tile's outputs
    __syncthreads();
    auto finish = [&](auto all) {
      constexpr bool PLAIN = decltype(all)::value;
      f32x2 sum[4];
      read8(sm.px[tid], sum);
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int v = tid + i * kBwdThreads, t = v / L::kRow, d = 8 * (v % L::kRow);
        if (v >= L::kVecs || (!PLAIN && (t >= nt || ch.first + d >= ch.end))) continue;
        const size_t out = static_cast<size_t>(row0 + t0 + t) * a.D + ch.first + d;
        const f32x2 one = both(1.f), minus = both(-1.f);
        f32x2 x[4], q[4], w[4], p[4], skip[4];
        read8(&sm.x[buf][t][d], x);
        read8(&sm.dy[buf][t][d], p);
        read8(&sm.g[t][d], q);
        read8(&sm.skip[d], skip);
        if (Z) {
          f32x2 z[4], y[4], dz[4];
          read8(&sm.z[buf][Z ? t : 0][d], z);
          read8(&sm.p[t][d], y);
          if (PLAIN || a.skip)
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = fma2(skip[j], x[j], y[j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // silu = z sg, its slope sg (1 + z (1 - sg)) = sg + silu (1 - sg)
            const f32x2 sg = sigmoid2(z[j]), act = mul2(z[j], sg);
            dz[j] = mul2(mul2(p[j], y[j]), fma2(act, fma2(sg, minus, one), sg));
            p[j] = mul2(p[j], act);
          }
          store_pairs(static_cast<T*>(a.dz) + out, dz);
        }
        f32x2 bias[4], u[4], dt[4], dx[4];
        read8(&sm.dt[buf][t][d], dt);
        read8(&sm.bias[d], bias);
        read8(&sm.u[t][d], u);
        read8(sm.r(t, d), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          dx[j] = mul2(u[j], q[j]);
          // (A2 is log2(e) A)
          w[j] = fma2(x[j], q[j], mul2(w[j], both(1.f / kLog2e)));
        }
        if (PLAIN || a.skip)
#pragma unroll
          for (int j = 0; j < 4; ++j) dx[j] = fma2(skip[j], p[j], dx[j]);
        if (PLAIN || a.softplus)
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = mul2(w[j], sigmoid2(add2(dt[j], bias[j])));
        store_pairs(static_cast<T*>(a.dx) + out, dx);
        store_pairs(static_cast<T*>(a.ddt) + out, w);
        write8(sm.r(t, d), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[j] = fma2(p[j], x[j], sum[j]);
      }
      write8(sm.px[tid], sum);
    };
    if (plain)
      finish(std::true_type{});
    else
      finish(std::false_type{});
    const int blocks = gridDim.x / a.G, block = blockIdx.x % blocks;
    for (int i = tid; i < nt * N / 2; i += kBwdThreads) {      // four sums each
      const int t = i / (N / 2), j = i % (N / 2) * 4;
      float4 s = *reinterpret_cast<const float4*>(sm.dbc(0, t) + j);
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(sm.dbc(w, t) + j);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
      }
      *reinterpret_cast<float4*>(
          sp.bc_part +
          (((static_cast<size_t>(block) * a.B + b) * a.T + t0 + t) * a.G + ch.group) * 2 * N + j) = s;
    }
    __syncthreads();
    if (a.dt_bias) {
#pragma unroll
      for (int i = 0; i < L::kSums; ++i) {
        const int d = tid + i * kBwdThreads;
        if (d >= L::kChannels) break;
        if (nt == kTile) {
#pragma unroll
          for (int t = 0; t < kTile; ++t) dbias[i] += *sm.r(t, d);
        } else {
          for (int t = 0; t < nt; ++t) dbias[i] += *sm.r(t, d);
        }
      }
    }
  }

  // (places of channels past the group's end are not written)
  if (live) {
    float4 v[4];
    from_items(dA, nx, v);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float4*>(sp.dA_part + at * state + place(i)) = v[i];
    if (from_start && a.dh0) {
      from_items(E, nx, v);
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<float4*>(a.dh0 + b * state + place(i)) = v[i];
    }
  }
#pragma unroll
  for (int i = 0; i < L::kSums; ++i) {
    const int d = tid + i * kBwdThreads;
    if (d >= L::kChannels || ch.first + d >= ch.end) continue;
    // dskip: threads kRow apart have the same channels
    float s = 0.f;
    for (int k = d / 8; k < kBwdThreads; k += L::kRow) s += sm.px[k][d % 8];
    sp.d_part[at * 2 * a.D + ch.first + d] = s;
    sp.d_part[(at * 2 + 1) * a.D + ch.first + d] = dbias[i];
  }
}

// Adds up the partial sums in a fixed order, four neighbouring ones a thread. The first CTAs
// take dA, dskip and ddt_bias, over batch rows and segments: 128 of them a CTA, every eighth row
// a warp (all rows in one thread's turn: 20 us for 4 x 4096 x 2048 x 16, two thirds of it these
// few threads' wait). The others take dBm and dCm, over the CTAs' channels.
constexpr int kSumThreads = 256, kSumWarps = kSumThreads / 32;

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
  return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

template <typename T>
__global__ void __launch_bounds__(kSumThreads)
    space_sums_kernel(const SpaceArgs a, const SpaceSplit sp, int first) {
  __shared__ float4 part[kSumWarps][32];
  const long long da = static_cast<long long>(a.D) * a.N;
  if (static_cast<int>(blockIdx.x) < first) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rows = a.B * sp.segments;
    const long long i = 4 * (32LL * blockIdx.x + lane), j = i - da;
    const bool live = j < 2 * a.D;
    const float* from = j < 0 ? sp.dA_part + i : sp.d_part + j;
    const long long stride = j < 0 ? da : 2LL * a.D;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live)
#pragma unroll 8
      for (int k = warp; k < rows; k += kSumWarps)
        s = add4(s, __ldcs(reinterpret_cast<const float4*>(from + k * stride)));
    part[warp][lane] = s;
    __syncthreads();
    if (warp > 0 || !live) return;
#pragma unroll
    for (int w = 1; w < kSumWarps; ++w) s = add4(s, part[w][lane]);
    float* out = j < 0       ? a.dA + i
                 : j < a.D ? (a.skip ? a.dskip + j : nullptr)
                           : (a.dt_bias ? a.ddt_bias + j - a.D : nullptr);
    if (out) *reinterpret_cast<float4*>(out) = s;
    return;
  }
  const long long bc = static_cast<long long>(a.B) * a.T * a.G * 2 * a.N;
  for (long long i = 4 * (static_cast<long long>(blockIdx.x - first) * kSumThreads + threadIdx.x);
       i < bc; i += 4LL * (gridDim.x - first) * kSumThreads) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 16
    for (int k = 0; k < sp.blocks; ++k)
      s = add4(s, __ldcs(reinterpret_cast<const float4*>(sp.bc_part + i + k * bc)));
    const int n = static_cast<int>(i % a.N), which = static_cast<int>(i / a.N % 2);
    T* out = static_cast<T*>(which ? a.dCm : a.dBm) + i / (2 * a.N) * a.N + n;
    store2(out, s.x, s.y);
    store2(out + 2, s.z, s.w);
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

int space_bwd_channels(int N, bool f32) { return bwd_warps(N, f32) * 4 * 32 / (N / 4); }

cudaError_t launch_space_bwd_states(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                                    cudaStream_t stream) {
  return by_states(a.N, f32, [&](auto t, auto n) {
    auto run = [&](auto cut) {
      constexpr auto kern = &space_bwd_states_kernel<decltype(t), n, cut>;
      constexpr int kBytes = static_cast<int>(sizeof(PreShared<decltype(t), n>));
      const cudaError_t err = allow_shared<kern, kBytes>();
      if (err != cudaSuccess) return err;
      kern<<<dim3(a.G * blocks_of(a, PreLayout<n>::kChannels), sp.segments, a.B), kThreads, kBytes,
             stream>>>(a, sp);
      return cudaGetLastError();
    };
    return sp.segments > 1 ? run(std::true_type{}) : run(std::false_type{});
  });
}

cudaError_t launch_space_bwd(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                             cudaStream_t stream) {
  const cudaError_t err = by_states(a.N, f32, [&](auto t, auto n) {
    auto run = [&](auto gated) {
      constexpr auto kern = &space_bwd_kernel<decltype(t), n, gated>;
      constexpr int kBytes = static_cast<int>(sizeof(BwdShared<decltype(t), n, gated>));
      const cudaError_t e = allow_shared<kern, kBytes>();
      if (e != cudaSuccess) return e;
      using L = BwdLayout<n, sizeof(decltype(t)) == 4>;
      kern<<<dim3(a.G * blocks_of(a, L::kChannels), sp.segments, a.B), L::kBwdThreads, kBytes,
             stream>>>(a, sp);
      return cudaGetLastError();
    };
    return a.z ? run(std::true_type{}) : run(std::false_type{});
  });
  if (err != cudaSuccess) return err;
  const int first = static_cast<int>((static_cast<long long>(a.D) * (a.N + 2) + 127) / 128);
  const long long want =      // the sums are a multiple of 16
      (static_cast<long long>(a.B) * a.T * a.G * 2 * a.N / 4 + kSumThreads - 1) / kSumThreads;
  const unsigned grid = first + static_cast<unsigned>(want < 152 * 32 ? want : 152 * 32);
  if (f32)
    space_sums_kernel<float><<<grid, kSumThreads, 0, stream>>>(a, sp, first);
  else
    space_sums_kernel<__nv_bfloat16><<<grid, kSumThreads, 0, stream>>>(a, sp, first);
  return cudaGetLastError();
}

}  // namespace gdr
