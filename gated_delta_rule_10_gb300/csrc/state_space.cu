// State space recurrence, forward: N states for each channel,
//   h_t[d,n] = exp(u_t[d] A[d,n]) h_{t-1}[d,n] + u_t[d] x_t[d] B_t[n]
//   y_t[d] = (sum_n C_t[n] h_t[d,n] + skip[d] x_t[d]) silu(z_t[d]),   u = softplus(dt + bias).
//
// Not a product of matrices: every (token, channel, state) has a decay of its own, so it is
// an exponential and four multiply-adds each, against 8 bytes of bf16 for a token and
// channel. What bounds it is the issue of instructions (62% of the slots), shared memory (61%)
// and the fp32 pipe (56%), not HBM (2 TB/s): 468 us for 4 x 4096 x 4096 channels x 16 bf16,
// 908 for 1 x 65536 x 2048. Multiply-adds run two to an instruction.
//
// Cut into segments, a thread holds 8 states of two channels and walks the tokens in order;
// N / 8 neighbouring lanes share the channels and add their parts of y. A tile of tokens is
// staged in shared memory as u and u x for each channel and B, C in fp32; the next tile's
// inputs are copied to shared memory meanwhile, without registers (prefetched in registers:
// 681 us for the first shape, then 583). With one channel a thread every B and C read from
// shared memory served half as many states: 714. A thread stages what it has copied itself,
// and takes y from where it has staged u. A warp stages the channels that it walks, so that only
// B and C, in two places in turn, need the CTA's barrier, one a tile (with two 1% more, 3% with
// 8 states); with 64 states, whose B and C take more room, and uncut it is two. Whole tiles are
// requested, staged and finished without branches (484 -> 468 us).
//
// Few sequences are cut into segments until the CTAs fill the SMs: a first launch walks all
// but the last one from zero for their end states and sums of u, a second chains them
// (exp(A sum u) is a whole segment's decay). Uncut, a thread has 4 states of one channel, so
// that there are four times the threads: the CTAs fill the SMs sooner, and short calls wait
// less (2 x 257 tokens x 192 channels: 18 us in one launch).
#include <type_traits>

#include "state_space.cuh"

namespace gdr {
namespace {

// NARROW: a thread has 4 states of one channel instead of 8 of two.
template <int N, bool NARROW>
struct Layout {
  static constexpr int kThreads = NARROW ? 256 : 128;
  static constexpr int kOwn = NARROW ? 1 : 2;                    // channels of a thread
  static constexpr int kStates = NARROW ? 4 : 8;                 // states of each
  static constexpr int kLanes = N / kStates;                     // lanes of a channel
  static constexpr int kChannels = kOwn * kThreads / kLanes;     // channels of a CTA
  // A warp stages the channels that it walks.
  static constexpr bool kApart = !NARROW && N < 64;
  static constexpr int kTile = NARROW || N == 64 ? 32 : N == 32 ? 16 : N;   // tokens of a tile
  static constexpr int kRow = (kApart ? kOwn * 32 / kLanes : kChannels) / 8;   // vectors of 8
  static constexpr int kVecs = kTile * kChannels / 8;            // vectors of 8 channels in a tile
  static constexpr int kPer = (kVecs + kThreads - 1) / kThreads;
  static constexpr int kBcVecs = 2 * kTile * N / 8;              // vectors of B and C
  static constexpr int kBcPer = (kBcVecs + kThreads - 1) / kThreads;
};

template <typename T, int N, bool NARROW>
struct __align__(16) Shared {
  using L = Layout<N, NARROW>;
  float u[L::kTile][L::kChannels], g[L::kTile][L::kChannels];    // u (then y), u x
  float bc[L::kApart ? 2 : 1][2][L::kTile][N];
  T x[2][L::kTile][L::kChannels], dt[L::kTile][L::kChannels], z[2][L::kTile][L::kChannels];
  T raw_bc[2][L::kTile][N];
  float bias[L::kChannels], skip[L::kChannels];
  unsigned starts[4];
};

// WALK: y and the end state, from the segment's start state. Else: the segment's own end
// state (segment 0's from h0), its sum of u and whether a document starts in it.
template <typename T, int N, bool NARROW, bool WALK>
__global__ void __launch_bounds__(NARROW ? 256 : 128,
                                  sizeof(T) == 2 ? (NARROW ? 2 : WALK ? 4 : 5) : (NARROW ? 1 : 2))
    space_kernel(const SpaceArgs a, const SpaceSplit sp) {
  using L = Layout<N, NARROW>;
  constexpr int kThreads = L::kThreads, kOwn = L::kOwn, kStates = L::kStates;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Shared<T, N, NARROW>& sm = *reinterpret_cast<Shared<T, N, NARROW>*>(raw_smem);
  const int tid = threadIdx.x;
  const Channels ch(a, L::kChannels, blockIdx.x);
  const int seg = blockIdx.y, b = blockIdx.z;
  const int t_begin = seg * sp.seg_len, t_end = min(t_begin + sp.seg_len, a.T);
  const long long row0 = static_cast<long long>(b) * a.T;

  // this thread's states
  const int lane = tid % L::kLanes, ci = kOwn * (tid / L::kLanes), c = ch.first + ci;
  const int n0 = lane * kStates;
  const bool live = c < ch.end;      // channels come in eights
  const bool busy = ch.first + kOwn * (tid / 32 * 32 / L::kLanes) < ch.end;   // this warp's any
  f32x2 A2[kOwn][kStates / 2], h[kOwn][kStates / 2];
  f32x2 usum = 0;                    // of the two channels
  const size_t state = static_cast<size_t>(a.D) * N;
  const float* from = nullptr;
  if (WALK && sp.segments > 1)
    from = sp.h + (static_cast<size_t>(b) * sp.segments + seg) * state;
  else if (seg == 0)
    from = a.h0 ? a.h0 + b * state : nullptr;
#pragma unroll
  for (int o = 0; o < kOwn; ++o) {
    const size_t own = static_cast<size_t>(c + o) * N + n0;     // in a [D, N] array
    f32x2 A[kStates / 2], v[kStates / 2];
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) A[i] = v[i] = 0;
    if (live) {
#pragma unroll
      for (int i = 0; i < kStates / 4; ++i) {
        const ulonglong2 q = __ldg(reinterpret_cast<const ulonglong2*>(a.A + own) + i);
        A[2 * i] = q.x;
        A[2 * i + 1] = q.y;
        if (from) {
          const ulonglong2 w = reinterpret_cast<const ulonglong2*>(from + own)[i];
          v[2 * i] = w.x;
          v[2 * i + 1] = w.y;
        }
        if (!WALK && seg == 0)
          reinterpret_cast<ulonglong2*>(sp.h + static_cast<size_t>(b) * sp.segments * state + own)[i] =
              make_ulonglong2(v[2 * i], v[2 * i + 1]);
      }
    }
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) {
      A2[o][i] = mul2(A[i], both(kLog2e));
      h[o][i] = v[i];
    }
  }
  for (int i = tid; i < L::kChannels; i += kThreads) {
    const int d = ch.first + i;
    sm.bias[i] = a.dt_bias && d < ch.end ? a.dt_bias[d] : 0.f;
    sm.skip[i] = a.skip && d < ch.end ? a.skip[d] : 0.f;
  }

  bool mark = false;
  // what a thread copies, stages and stores: vectors of 8 channels of a tile's tokens
  const int first = L::kApart ? tid % 32 : tid, step = L::kApart ? 32 : kThreads;
  const int wide = L::kApart ? tid / 32 * (8 * L::kRow) : 0;
  auto token_of = [&](int i) { return (first + i * step) / L::kRow; };
  auto channel_of = [&](int i) { return wide + 8 * ((first + i * step) % L::kRow); };
  // copies a tile's inputs: x, dt and z, B and C; `k` of two places for what the tile's end needs
  const bool full = ch.first + L::kChannels <= ch.end;
  auto fetch = [&](int t0, int k) {
    auto copies = [&](auto plain) {      // PLAIN: nothing of the tile is missing
      constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int t = token_of(i), d = channel_of(i);
        if (t < L::kTile && (PLAIN || (t0 + t < t_end && ch.first + d < ch.end))) {
          const long long row = row0 + t0 + t;
          copy8(&sm.x[k][t][d], static_cast<const T*>(a.x) + row * a.xs + ch.first + d);
          copy8(&sm.dt[t][d], static_cast<const T*>(a.dt) + row * a.dts + ch.first + d);
          if (WALK && a.z)
            copy8(&sm.z[k][t][d], static_cast<const T*>(a.z) + row * a.zs + ch.first + d);
        }
      }
#pragma unroll
      for (int i = 0; i < L::kBcPer; ++i) {
        const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
        const int t = w / (N / 8), n = 8 * (w % (N / 8));
        if (v < (WALK ? L::kBcVecs : L::kBcVecs / 2) && (PLAIN || t0 + t < t_end))
          copy8(&sm.raw_bc[which][t][n],
                (which ? static_cast<const T*>(a.Cm) + (row0 + t0 + t) * a.cs
                       : static_cast<const T*>(a.Bm) + (row0 + t0 + t) * a.bs) +
                    ch.group * N + n);
      }
    };
    if (full && t0 + L::kTile <= t_end)
      copies(std::true_type{});
    else
      copies(std::false_type{});
    mark = a.starts && tid < L::kTile && t0 + tid < t_end && a.starts[row0 + t0 + tid] != 0;
  };
  // what this thread has copied, as the walk reads it
  auto stage = [&](int t0, int k) {
    copies_done();
    // PLAIN: nothing of the tile is missing and u is a softplus, so that no branch parts the
    // vectors' long chains
    auto steps = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int t = token_of(i), d = channel_of(i);
        if (t >= L::kTile) break;
        f32x2 x[4], u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = u[j] = 0;
        if (PLAIN || (t0 + t < t_end && ch.first + d < ch.end)) {
          f32x2 bias[4];
          read8(&sm.x[k][t][d], x);
          read8(&sm.dt[t][d], u);
          read8(&sm.bias[d], bias);
#pragma unroll
          for (int j = 0; j < 4; ++j) u[j] = add2(u[j], bias[j]);
          if (PLAIN || a.softplus)
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = softplus2(u[j]);
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = mul2(u[j], x[j]);
        }
        write8(&sm.u[t][d], u);
        write8(&sm.g[t][d], x);
      }
    };
    if (full && a.softplus && t0 + L::kTile <= t_end)
      steps(std::true_type{});
    else
      steps(std::false_type{});
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = w / (N / 8), n = 8 * (w % (N / 8));
      if (v >= (WALK ? L::kBcVecs : L::kBcVecs / 2)) break;
      f32x2 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = 0;
      if (t0 + t < t_end) read8(&sm.raw_bc[which][t][n], x);
      write8(&sm.bc[L::kApart ? k : 0][which][t][n], x);
    }
    const unsigned m = __ballot_sync(0xffffffffu, mark);
    if (tid == 0) sm.starts[L::kApart ? k : 0] = m;
  };

  int cleared = 0;
  // one token, which may be a document's first: this thread's parts of its channels' y
  auto token = [&](int k, int t, bool first, float (&y)[kOwn]) {
    float u[kOwn], g[kOwn];
    if constexpr (kOwn == 2) {
      const float2 v = *reinterpret_cast<const float2*>(&sm.u[t][ci]);
      const float2 w = *reinterpret_cast<const float2*>(&sm.g[t][ci]);
      u[0] = v.x; u[1] = v.y; g[0] = w.x; g[1] = w.y;
      if (!WALK) usum = add2(usum, pair(v.x, v.y));
    } else {
      u[0] = sm.u[t][ci];
      g[0] = sm.g[t][ci];
      if (!WALK) usum = add2(usum, pair(u[0], 0.f));
    }
    if (first) {
#pragma unroll
      for (int o = 0; o < kOwn; ++o)
#pragma unroll
        for (int i = 0; i < kStates / 2; ++i) h[o][i] = 0;
    }
    const ulonglong2* B = reinterpret_cast<const ulonglong2*>(&sm.bc[k][0][t][n0]);
    const ulonglong2* C = reinterpret_cast<const ulonglong2*>(&sm.bc[k][1][t][n0]);
    f32x2 part[kOwn];
#pragma unroll
    for (int q = 0; q < kStates / 4; ++q) {
      const ulonglong2 bq = B[q];
      ulonglong2 cq;
      if (WALK) cq = C[q];
#pragma unroll
      for (int o = 0; o < kOwn; ++o) {
        const f32x2 u2 = both(u[o]), g2 = both(g[o]);
        f32x2& h0 = h[o][2 * q];
        f32x2& h1 = h[o][2 * q + 1];
        h0 = fma2(g2, bq.x, mul2(decay2(A2[o][2 * q], u2), h0));
        h1 = fma2(g2, bq.y, mul2(decay2(A2[o][2 * q + 1], u2), h1));
        if (WALK) part[o] = fma2(cq.y, h1, q ? fma2(cq.x, h0, part[o]) : mul2(cq.x, h0));
      }
    }
    if (WALK)
#pragma unroll
      for (int o = 0; o < kOwn; ++o) y[o] = sum2(part[o]);
  };
  // y of four tokens: summed over the channels' lanes by halves, each lane going on with half
  // of the sums (one of two channels, half of the tokens). Written behind all four, whose
  // loads would else wait for one another.
  auto put = [&](int t, const float (&y)[4][kOwn]) {
    // `n` sums, of which lanes apart by `bit` keep every other one: index 2 i + (lane & bit)
    auto halve = [&](auto n, const float* in, int bit, float* out) {
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const bool up = lane & bit;
        out[i] = (up ? in[2 * i + 1] : in[2 * i]) +
                 __shfl_xor_sync(0xffffffffu, up ? in[2 * i] : in[2 * i + 1], bit);
      }
    };
    using std::integral_constant;
    if constexpr (L::kLanes == 1) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int o = 0; o < kOwn; ++o) sm.u[t + k][ci + o] = y[k][o];
    } else {
      constexpr int kAll = 4 * kOwn;           // 8 or 4 sums, the channels fastest
      float r[kAll / 2], q[kAll / 4 > 0 ? kAll / 4 : 1], v[1];
      halve(integral_constant<int, kAll>{}, &y[0][0], 1, r);
      const int b0 = lane & 1, b1 = (lane >> 1) & 1, b2 = (lane >> 2) & 1;
      auto at = [&](int i) -> float& { return sm.u[t + i / kOwn][ci + i % kOwn]; };
      if constexpr (L::kLanes == 2) {
#pragma unroll
        for (int i = 0; i < kAll / 2; ++i) at(2 * i + b0) = r[i];
      } else {
        halve(integral_constant<int, kAll / 2>{}, r, 2, q);
        if constexpr (L::kLanes == 4) {
#pragma unroll
          for (int i = 0; i < kAll / 4; ++i) at(4 * i + 2 * b1 + b0) = q[i];
        } else if constexpr (kAll == 8) {      // 8 lanes of two channels
          halve(integral_constant<int, 2>{}, q, 4, v);
          at(4 * b2 + 2 * b1 + b0) = v[0];
        } else {                               // 8 or 16 lanes of one: whole
          v[0] = q[0] + __shfl_xor_sync(0xffffffffu, q[0], 4);
          if constexpr (L::kLanes == 16) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 8);
          if (lane < 4) at(2 * b1 + b0) = v[0];
        }
      }
    }
  };

  fetch(t_begin, 0);
  __syncthreads();
  stage(t_begin, 0);
  __syncthreads();
  int k = 0;      // the tile's place
  for (int t0 = t_begin; t0 < t_end; t0 += L::kTile, k ^= 1) {
    fetch(t0 + L::kTile, k ^ 1);
    const int nt = min(L::kTile, t_end - t0);
    const int place = L::kApart ? k : 0;
    const unsigned starts = sm.starts[place];
    // (tokens behind the end have u = B = C = 0 and leave the states as they are)
    if (NARROW && !busy) {      // (a test that costs the cut calls 1%)
    } else if (starts == 0 && nt == L::kTile) {
      if constexpr (NARROW) {
        // y of four tokens is written behind the next four, whose loads need not wait for it
        // (few warps: 2 x 257 tokens x 192 channels 20.1 -> 17.9 us; with more it costs 0.5%)
        float y[2][4][kOwn];
#pragma unroll
        for (int t = 0; t < L::kTile; t += 4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) token(0, t + j, false, y[t / 4 % 2][j]);
          if (t > 0) put(t - 4, y[(t / 4 + 1) % 2]);
        }
        put(L::kTile - 4, y[(L::kTile / 4 + 1) % 2]);
      } else {
        // (N = 16 bf16 1% faster unrolled whole, fp32 4% slower)
        constexpr int kAhead = sizeof(T) == 2 && L::kTile <= 16 ? 4 : 2;
#pragma unroll kAhead
        for (int t = 0; t < L::kTile; t += 4) {
          float y[4][kOwn];
#pragma unroll
          for (int j = 0; j < 4; ++j) token(place, t + j, false, y[j]);
          if (WALK) put(t, y);
        }
      }
    } else {
      for (int t = 0; t < nt; t += 4) {
        float y[4][kOwn];
#pragma unroll
        for (int j = 0; j < 4; ++j) token(place, t + j, (starts >> (t + j)) & 1, y[j]);
        if (WALK) put(t, y);
      }
    }
    cleared |= starts != 0;
    if (L::kApart)
      __syncwarp();
    else
      __syncthreads();
    auto finish = [&](auto plain) {
      constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int t = token_of(i), d = channel_of(i);
        if (t >= L::kTile || (!PLAIN && (t0 + t >= t_end || ch.first + d >= ch.end))) continue;
        f32x2 x[4], z[4], skip[4], y[4];
        read8(&sm.u[t][d], y);
        if (PLAIN || a.skip) {
          read8(&sm.x[k][t][d], x);
          read8(&sm.skip[d], skip);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = fma2(skip[j], x[j], y[j]);
        }
        if (PLAIN || a.z) {
          read8(&sm.z[k][t][d], z);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = mul2(y[j], mul2(z[j], sigmoid2(z[j])));
        }
        store_pairs(static_cast<T*>(a.y) + (row0 + t0 + t) * a.D + ch.first + d, y);
      }
    };
    if (WALK) {
      if (full && nt == L::kTile && a.skip && a.z)
        finish(std::true_type{});
      else
        finish(std::false_type{});
    }
    if (t0 + L::kTile < t_end) {
      stage(t0 + L::kTile, k ^ 1);
      __syncthreads();
    }
  }

  float* out = nullptr;
  if (WALK) {
    if (seg == sp.segments - 1 && a.hT) out = a.hT + b * state;
  } else {
    out = sp.h + (static_cast<size_t>(b) * sp.segments + seg + 1) * state;
    float u0, u1;
    split(usum, u0, u1);
    float* total = sp.total + (static_cast<size_t>(b) * sp.segments + seg) * a.D + c;
    if (live && n0 == 0) {
      total[0] = u0;
      if (kOwn == 2) total[1] = u1;
    }
    if (blockIdx.x == 0 && tid == 0) sp.cleared[b * sp.segments + seg] = cleared;
  }
  if (out && live) {
#pragma unroll
    for (int o = 0; o < kOwn; ++o) {
      ulonglong2* p = reinterpret_cast<ulonglong2*>(out + static_cast<size_t>(c + o) * N + n0);
#pragma unroll
      for (int i = 0; i < kStates / 4; ++i) p[i] = make_ulonglong2(h[o][2 * i], h[o][2 * i + 1]);
    }
  }
}

constexpr int kFlatThreads = 256;    // of the kernels below

// The start states of the segments, chained: slot s of `sp.h` from what segment s - 1 alone
// adds (for slots 0 and 1 whole already), in place; and with `blockIdx.y` the gradients that
// reach the segments' ends, from the last one on. A segment's decay is exp(A sum u), none of
// a state passes a document's start. Four states a thread; loads of kBatch segments at once.
__global__ void __launch_bounds__(kFlatThreads) space_chain_kernel(const SpaceArgs a,
                                                               const SpaceSplit sp) {
  constexpr int kBatch = 8;
  const long long id = static_cast<long long>(blockIdx.x) * kFlatThreads + threadIdx.x;
  const long long state = static_cast<long long>(a.D) * a.N;
  if (id >= a.B * state / 4) return;
  const int b = static_cast<int>(id / (state / 4)), S = sp.segments;
  const long long own = id % (state / 4) * 4;
  const int d = static_cast<int>(own / a.N);
  const bool back = blockIdx.y == 1;
  const float4 A = *reinterpret_cast<const float4*>(a.A + own);
  const float A2[4] = {A.x * kLog2e, A.y * kLog2e, A.z * kLog2e, A.w * kLog2e};
  float* slots = (back ? sp.e : sp.h) + static_cast<long long>(b) * S * state + own;
  // step i: slot(i) <- slot(i) + decay of segment(i) * slot(i - 1)
  auto slot = [&](int i) { return back ? S - 2 - i : 1 + i; };
  auto segment = [&](int i) { return back ? S - 1 - i : i; };
  const int steps = S - 1;
  float4 v = *reinterpret_cast<const float4*>(slots + slot(0) * state);
  for (int i = 1; i < steps; i += kBatch) {
    float4 w[kBatch];
    float u[kBatch];
    int gone[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k < steps) {
        w[k] = *reinterpret_cast<const float4*>(slots + slot(i + k) * state);
        u[k] = sp.total[(static_cast<long long>(b) * S + segment(i + k)) * a.D + d];
        gone[k] = sp.cleared[b * S + segment(i + k)];
      }
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i + k < steps) {
        if (gone[k]) {
          v = w[k];
        } else {
          v.x = fmaf(exp2_fast(A2[0] * u[k]), v.x, w[k].x);
          v.y = fmaf(exp2_fast(A2[1] * u[k]), v.y, w[k].y);
          v.z = fmaf(exp2_fast(A2[2] * u[k]), v.z, w[k].z);
          v.w = fmaf(exp2_fast(A2[3] * u[k]), v.w, w[k].w);
        }
        *reinterpret_cast<float4*>(slots + slot(i + k) * state) = v;
      }
  }
}

// One token of each sequence: the states are read and written once, which is all there is to
// do. A warp has 32 channels of a sequence: a lane makes the step size of one of them, then
// N / 4 neighbouring lanes have four states each of 128 / N channels at a time, whose loads
// are requested four rounds at once. (A channel's lanes that each made its step size: 39 us
// for 256 x 4096 x 16, bound by instructions.)
template <typename T>
__device__ __forceinline__ float4 read4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return __ldg(reinterpret_cast<const float4*>(p));
  } else {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  }
}

template <typename T, int N>
__global__ void __launch_bounds__(kFlatThreads) space_step_kernel(const SpaceArgs a, int blocks,
                                                                  long long warps) {
  constexpr int kLanes = N / 4, kRound = 32 / kLanes;      // channels of a round
  constexpr int kTogether = kLanes < 4 ? kLanes : 4;
  const long long w = static_cast<long long>(blockIdx.x) * (kFlatThreads / 32) + threadIdx.x / 32;
  if (w >= warps) return;
  const int lane = threadIdx.x & 31, d0 = static_cast<int>(w % blocks) * 32, mine = d0 + lane;
  const long long b = w / blocks;
  const int sub = lane / kLanes, n = lane % kLanes * 4, each = a.D / a.G;
  float* hp = a.hT + b * a.D * N;
  float u = 0.f, x = 0.f, z = 0.f;
  if (mine < a.D) {
    x = static_cast<float>(static_cast<const T*>(a.x)[b * a.xs + mine]);
    u = static_cast<float>(static_cast<const T*>(a.dt)[b * a.dts + mine]);
    if (a.z) z = static_cast<float>(static_cast<const T*>(a.z)[b * a.zs + mine]);
  }
  float y = 0.f;
  float4 h[kTogether], A[kTogether];
#pragma unroll
  for (int r0 = 0; r0 < kLanes; r0 += kTogether) {
#pragma unroll
    for (int r = 0; r < kTogether; ++r) {
      const int d = d0 + (r0 + r) * kRound + sub;
      if (d < a.D) {
        h[r] = __ldcs(reinterpret_cast<const float4*>(hp + static_cast<size_t>(d) * N + n));
        A[r] = __ldg(reinterpret_cast<const float4*>(a.A + static_cast<size_t>(d) * N + n));
      }
    }
    if (r0 == 0 && mine < a.D) {      // the states are on their way
      if (a.dt_bias) u += a.dt_bias[mine];
      if (a.softplus) u = softplus(u);
    }
#pragma unroll
    for (int r = 0; r < kTogether; ++r) {
      const int from = (r0 + r) * kRound + sub, d = d0 + from;
      const float ud = __shfl_sync(0xffffffffu, u, from), xd = __shfl_sync(0xffffffffu, x, from);
      float s = 0.f;
      if (d < a.D) {
        const int group = d / each;
        const float4 B = read4(static_cast<const T*>(a.Bm) + b * a.bs + group * N + n);
        const float4 C = read4(static_cast<const T*>(a.Cm) + b * a.cs + group * N + n);
        const f32x2 v = both(kLog2e * ud), g = both(ud * xd);
        const f32x2 lo = fma2(g, pair(B.x, B.y),
                              mul2(decay2(pair(A[r].x, A[r].y), v), pair(h[r].x, h[r].y)));
        const f32x2 hi = fma2(g, pair(B.z, B.w),
                              mul2(decay2(pair(A[r].z, A[r].w), v), pair(h[r].z, h[r].w)));
        split(lo, h[r].x, h[r].y);
        split(hi, h[r].z, h[r].w);
        s = fmaf(C.x, h[r].x, fmaf(C.y, h[r].y, fmaf(C.z, h[r].z, C.w * h[r].w)));
        __stcs(reinterpret_cast<float4*>(hp + static_cast<size_t>(d) * N + n), h[r]);
      }
#pragma unroll
      for (int off = 1; off < kLanes; off *= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
      // to the lane that has the channel
      const float got = __shfl_sync(0xffffffffu, s, (lane % kRound) * kLanes);
      if (lane / kRound == r0 + r) y = got;
    }
  }
  if (mine < a.D) {
    if (a.skip) y = fmaf(a.skip[mine], x, y);
    if (a.z) y *= silu(z);
    static_cast<T*>(a.y)[b * a.D + mine] = static_cast<T>(y);
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

template <bool NARROW, bool WALK>
cudaError_t launch_as(const SpaceArgs& a, const SpaceSplit& sp, int segments, bool f32,
                      cudaStream_t stream) {
  return by_states(a.N, f32, [&](auto t, auto n) {
    using L = Layout<n, NARROW>;
    constexpr int kBytes = static_cast<int>(sizeof(Shared<decltype(t), n, NARROW>));
    constexpr auto kern = &space_kernel<decltype(t), n, NARROW, WALK>;
    const cudaError_t err = allow_shared<kern, kBytes>();
    if (err != cudaSuccess) return err;
    const int each = a.D / a.G, per = (each + L::kChannels - 1) / L::kChannels;
    kern<<<dim3(a.G * per, segments, a.B), L::kThreads, kBytes, stream>>>(a, sp);
    return cudaGetLastError();
  });
}

}  // namespace

int space_channels(int N, bool narrow) {
  return narrow ? 256 / (N / 4) : 2 * 128 / (N / 8);
}
cudaError_t launch_space_states(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                                cudaStream_t stream) {
  return launch_as<false, false>(a, sp, sp.segments - 1, f32, stream);
}
cudaError_t launch_space_walk(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                              cudaStream_t stream) {
  return sp.segments == 1 ? launch_as<true, true>(a, sp, 1, f32, stream)
                          : launch_as<false, true>(a, sp, sp.segments, f32, stream);
}
cudaError_t launch_space_chain(const SpaceArgs& a, const SpaceSplit& sp, bool backward,
                               cudaStream_t stream) {
  if (sp.segments < 3) return cudaSuccess;     // nothing to add
  const long long total = static_cast<long long>(a.B) * a.D * (a.N / 4);
  const long long grid = (total + kFlatThreads - 1) / kFlatThreads;
  if (grid > 2147483647LL) return cudaErrorInvalidValue;
  space_chain_kernel<<<dim3(static_cast<unsigned>(grid), backward ? 2 : 1), kFlatThreads, 0, stream>>>(
      a, sp);
  return cudaGetLastError();
}
cudaError_t launch_space_step(const SpaceArgs& a, bool f32, cudaStream_t stream) {
  const int blocks = (a.D + 31) / 32;
  const long long warps = static_cast<long long>(a.B) * blocks;
  const long long grid = (warps + kFlatThreads / 32 - 1) / (kFlatThreads / 32);
  if (grid > 2147483647LL) return cudaErrorInvalidValue;
  return by_states(a.N, f32, [&](auto t, auto n) {
    space_step_kernel<decltype(t), n>
        <<<static_cast<unsigned>(grid), kFlatThreads, 0, stream>>>(a, blocks, warps);
    return cudaGetLastError();
  });
}

}  // namespace gdr
