// State space recurrence, forward: N states for each channel,
//   h_t[d,n] = exp(u_t[d] A[d,n]) h_{t-1}[d,n] + u_t[d] x_t[d] B_t[n]
//   y_t[d] = (sum_n C_t[n] h_t[d,n] + skip[d] x_t[d]) silu(z_t[d]),   u = softplus(dt + bias).
//
// Not a product of matrices: every (token, channel, state) has a decay of its own, so it is
// an exponential and four multiply-adds each, against 8 bytes of bf16 for a token and
// channel. What bounds it is the exponential unit and the fp32 pipe; multiply-adds run two
// to an instruction.
//
// A thread holds 8 states of one channel and walks the tokens in order; N / 8 neighbouring
// lanes share a channel and add their parts of y. A tile of tokens is staged in shared
// memory as (u, u x) for each channel and B, C in fp32; the next tile's loads are in flight
// during the walk. The thread that writes a place's (u, u x) is the one that takes y from
// there, so that two barriers a tile are enough.
//
// Few sequences are cut into segments until the CTAs fill the SMs: a first launch walks all
// but the last one from zero for their end states and sums of u; a segment's CTA then
// chains those before it (exp(A sum u) is a whole segment's decay).
#include <type_traits>

#include "state_space.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kStates = 8;        // states of a thread

template <int N>
struct Layout {
  static constexpr int kLanes = N / kStates;              // lanes of a channel
  static constexpr int kChannels = kThreads / kLanes;     // channels of a CTA
  static constexpr int kTile = N == 8 ? 16 : 32;          // tokens of a tile
  static constexpr int kVecs = kTile * kChannels / 8;     // vectors of 8 channels in a tile
  static constexpr int kPer = (kVecs + kThreads - 1) / kThreads;
  static constexpr int kBcVecs = 2 * kTile * N / 8;       // vectors of B and C
  static constexpr int kBcPer = (kBcVecs + kThreads - 1) / kThreads;
};

template <int N>
struct __align__(16) Shared {
  float2 ug[Layout<N>::kTile][Layout<N>::kChannels];
  float bc[2][Layout<N>::kTile][N];
  float bias[Layout<N>::kChannels], skip[Layout<N>::kChannels];
  unsigned starts[4];
};

// WALK: y and the end state, from the segment's start state. Else: the segment's own end
// state (segment 0's from h0), its sum of u and whether a document starts in it.
template <typename T, int N, bool WALK>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1)
    space_kernel(const SpaceArgs a, const SpaceSplit sp) {
  using L = Layout<N>;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Shared<N>& sm = *reinterpret_cast<Shared<N>*>(raw_smem);
  const int tid = threadIdx.x;
  const Channels ch(a, L::kChannels, blockIdx.x);
  const int seg = blockIdx.y, b = blockIdx.z;
  const int t_begin = seg * sp.seg_len, t_end = min(t_begin + sp.seg_len, a.T);
  const long long row0 = static_cast<long long>(b) * a.T;

  // this thread's states
  const int c = ch.first + tid / L::kLanes, n0 = (tid % L::kLanes) * kStates;
  const bool live = c < ch.end;
  f32x2 A2[kStates / 2], h[kStates / 2];
  float usum = 0.f;
  const size_t state = static_cast<size_t>(a.D) * N;
  const size_t own = static_cast<size_t>(c) * N + n0;     // in a [D, N] array
  {
    float A[kStates], v[kStates];
#pragma unroll
    for (int i = 0; i < kStates; ++i) A[i] = v[i] = 0.f;
    if (live) {
      load8(a.A + own, A);
#pragma unroll
      for (int i = 0; i < kStates; ++i) A[i] *= kLog2e;
      if (WALK && sp.segments > 1) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float Aq[4] = {A[4 * q], A[4 * q + 1], A[4 * q + 2], A[4 * q + 3]};
          float hq[4];
          chain_states(a, sp, b, seg, c, n0 + 4 * q, Aq, hq);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * q + i] = hq[i];
        }
      } else if (seg == 0 && a.h0) {
        const float4* p = reinterpret_cast<const float4*>(a.h0 + b * state + own);
        const float4 lo = p[0], hi = p[1];
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
      }
      if (!WALK && seg == 0)
        store8(sp.h + static_cast<size_t>(b) * sp.segments * state + own, v);
    }
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) {
      A2[i] = pair(A[2 * i], A[2 * i + 1]);
      h[i] = pair(v[2 * i], v[2 * i + 1]);
    }
  }
  for (int i = tid; i < L::kChannels; i += kThreads) {
    const int d = ch.first + i;
    sm.bias[i] = a.dt_bias && d < ch.end ? a.dt_bias[d] : 0.f;
    sm.skip[i] = a.skip && d < ch.end ? a.skip[d] : 0.f;
  }

  Raw8<T> rx[L::kPer], rdt[L::kPer], rz[L::kPer], rbc[L::kBcPer];
  bool mark = false;
  // requests a tile: x and dt, B and C, the starts
  auto fetch = [&](int t0) {
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kThreads, t = t0 + v / (L::kChannels / 8);
      const int d = ch.first + 8 * (v % (L::kChannels / 8));
      if (v < L::kVecs && t < t_end && d < ch.end) {
        rx[i].load(static_cast<const T*>(a.x) + (row0 + t) * a.xs + d);
        rdt[i].load(static_cast<const T*>(a.dt) + (row0 + t) * a.dts + d);
      }
    }
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      const int t = t0 + w / (N / 8), n = 8 * (w % (N / 8));
      rbc[i].zero();
      if (v < (WALK ? L::kBcVecs : L::kBcVecs / 2) && t < t_end)
        rbc[i].load((which ? static_cast<const T*>(a.Cm) + (row0 + t) * a.cs
                           : static_cast<const T*>(a.Bm) + (row0 + t) * a.bs) +
                    ch.group * N + n);
    }
    mark = a.starts && tid < L::kTile && t0 + tid < t_end && a.starts[row0 + t0 + tid] != 0;
  };
  // and writes it to shared memory
  auto stage = [&](int t0) {
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) {
      const int v = tid + i * kThreads, t = v / (L::kChannels / 8);
      const int d = 8 * (v % (L::kChannels / 8));
      if (v >= L::kVecs) break;
      float x[8], u[8];
      if (t0 + t < t_end && ch.first + d < ch.end) {
        rx[i].get(x);
        rdt[i].get(u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u[j] += sm.bias[d + j];
          if (a.softplus) u[j] = softplus(u[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = u[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<float4*>(&sm.ug[t][d + 2 * j]) =
            make_float4(u[2 * j], u[2 * j] * x[2 * j], u[2 * j + 1], u[2 * j + 1] * x[2 * j + 1]);
    }
#pragma unroll
    for (int i = 0; i < L::kBcPer; ++i) {
      const int v = tid + i * kThreads, which = v / (L::kBcVecs / 2), w = v % (L::kBcVecs / 2);
      if (v >= (WALK ? L::kBcVecs : L::kBcVecs / 2)) break;
      float x[8];
      rbc[i].get(x);
      float4* p = reinterpret_cast<float4*>(&sm.bc[which][w / (N / 8)][8 * (w % (N / 8))]);
      p[0] = make_float4(x[0], x[1], x[2], x[3]);
      p[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
    const unsigned m = __ballot_sync(0xffffffffu, mark);
    if (tid == 0) sm.starts[0] = m;
  };

  int cleared = 0;
  // one token; FIRST: it may begin a document
  auto token = [&](int t, bool first) {
    const float2 ug = sm.ug[t][tid / L::kLanes];
    if (first) {
#pragma unroll
      for (int i = 0; i < kStates / 2; ++i) h[i] = pair(0.f, 0.f);
    }
    if (!WALK) usum += ug.x;
    const f32x2 u2 = pair(ug.x, ug.x), g2 = pair(ug.y, ug.y);
    const ulonglong2* B = reinterpret_cast<const ulonglong2*>(&sm.bc[0][t][n0]);
    const ulonglong2* C = reinterpret_cast<const ulonglong2*>(&sm.bc[1][t][n0]);
    f32x2 y = pair(0.f, 0.f);
#pragma unroll
    for (int q = 0; q < kStates / 4; ++q) {
      const ulonglong2 bq = B[q];
      h[2 * q] = fma2(exp2_pair(mul2(A2[2 * q], u2)), h[2 * q], mul2(g2, bq.x));
      h[2 * q + 1] = fma2(exp2_pair(mul2(A2[2 * q + 1], u2)), h[2 * q + 1], mul2(g2, bq.y));
      if (WALK) {
        const ulonglong2 cq = C[q];
        y = fma2(cq.x, h[2 * q], y);
        y = fma2(cq.y, h[2 * q + 1], y);
      }
    }
    if (WALK) {
      float s = sum2(y);
#pragma unroll
      for (int off = 1; off < L::kLanes; off *= 2) s += __shfl_xor_sync(0xffffffffu, s, off);
      if (tid % L::kLanes == 0) sm.ug[t][tid / L::kLanes].x = s;
    }
  };

  fetch(t_begin);
  __syncthreads();
  stage(t_begin);
  __syncthreads();
  for (int t0 = t_begin; t0 < t_end; t0 += L::kTile) {
    Raw8<T> cx[L::kPer];
#pragma unroll
    for (int i = 0; i < L::kPer; ++i) cx[i] = rx[i];
    if (WALK && a.z)
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int v = tid + i * kThreads, t = t0 + v / (L::kChannels / 8);
        const int d = ch.first + 8 * (v % (L::kChannels / 8));
        if (v < L::kVecs && t < t_end && d < ch.end)
          rz[i].load(static_cast<const T*>(a.z) + (row0 + t) * a.zs + d);
      }
    fetch(t0 + L::kTile);
    const int nt = min(L::kTile, t_end - t0);
    const unsigned starts = sm.starts[0];
    if (starts == 0 && nt == L::kTile) {
#pragma unroll 4
      for (int t = 0; t < L::kTile; ++t) token(t, false);
    } else {
      for (int t = 0; t < nt; ++t) token(t, (starts >> t) & 1);
      cleared |= starts != 0;
    }
    __syncthreads();
    if (WALK) {
#pragma unroll
      for (int i = 0; i < L::kPer; ++i) {
        const int v = tid + i * kThreads, t = v / (L::kChannels / 8);
        const int d = 8 * (v % (L::kChannels / 8));
        if (v >= L::kVecs || t0 + t >= t_end || ch.first + d >= ch.end) continue;
        float x[8], z[8], y[8];
        cx[i].get(x);
        if (a.z) rz[i].get(z);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          y[j] = sm.ug[t][d + j].x;
          if (a.skip) y[j] = fmaf(sm.skip[d + j], x[j], y[j]);
          if (a.z) y[j] *= silu(z[j]);
        }
        store8(static_cast<T*>(a.y) + (row0 + t0 + t) * a.D + ch.first + d, y);
      }
    }
    if (t0 + L::kTile < t_end) {
      stage(t0 + L::kTile);
      __syncthreads();
    }
  }

  float* out = nullptr;
  if (WALK) {
    if (seg == sp.segments - 1 && a.hT) out = a.hT + b * state;
  } else {
    out = sp.h + (static_cast<size_t>(b) * sp.segments + seg + 1) * state;
    if (live && n0 == 0) sp.total[(static_cast<size_t>(b) * sp.segments + seg) * a.D + c] = usum;
    if (blockIdx.x == 0 && tid == 0) sp.cleared[b * sp.segments + seg] = cleared;
  }
  if (out && live) {
    float v[kStates];
#pragma unroll
    for (int i = 0; i < kStates / 2; ++i) split(h[i], v[2 * i], v[2 * i + 1]);
    float4* p = reinterpret_cast<float4*>(out + own);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// One token of each sequence: the states are read and written once. A thread has four
// states of a channel, N / 4 neighbouring lanes a channel.
template <typename T, int N>
__global__ void __launch_bounds__(kThreads) space_step_kernel(const SpaceArgs a, long long total) {
  constexpr int kLanes = N / 4;
  const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const bool live = id < total;
  const long long bd = live ? id / kLanes : 0;
  const int d = static_cast<int>(bd % a.D), n = static_cast<int>(id % kLanes) * 4;
  const long long b = bd / a.D;
  float* hp = a.hT + bd * N + n;
  float y = 0.f, x = 0.f;
  if (live) {
    const float4 h4 = __ldcs(reinterpret_cast<const float4*>(hp));
    const float4 A4 = __ldg(reinterpret_cast<const float4*>(a.A + static_cast<long long>(d) * N + n));
    x = static_cast<float>(static_cast<const T*>(a.x)[b * a.xs + d]);
    float u = static_cast<float>(static_cast<const T*>(a.dt)[b * a.dts + d]);
    if (a.dt_bias) u += a.dt_bias[d];
    if (a.softplus) u = softplus(u);
    const float g = u * x;
    const int group = d / (a.D / a.G);
    const T* B = static_cast<const T*>(a.Bm) + b * a.bs + group * N + n;
    const T* C = static_cast<const T*>(a.Cm) + b * a.cs + group * N + n;
    float h[4] = {h4.x, h4.y, h4.z, h4.w};
    const float A[4] = {A4.x, A4.y, A4.z, A4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(exp2_fast(kLog2e * A[i] * u), h[i], g * static_cast<float>(B[i]));
      y = fmaf(static_cast<float>(C[i]), h[i], y);
    }
    __stcs(reinterpret_cast<float4*>(hp), make_float4(h[0], h[1], h[2], h[3]));
  }
#pragma unroll
  for (int off = 1; off < kLanes; off *= 2) y += __shfl_xor_sync(0xffffffffu, y, off);
  if (live && n == 0) {
    if (a.skip) y = fmaf(a.skip[d], x, y);
    if (a.z) y *= silu(static_cast<float>(static_cast<const T*>(a.z)[b * a.zs + d]));
    static_cast<T*>(a.y)[bd] = static_cast<T>(y);
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

template <bool WALK>
cudaError_t launch(const SpaceArgs& a, const SpaceSplit& sp, int segments, bool f32,
                   cudaStream_t stream) {
  return by_states(a.N, f32, [&](auto t, auto n) {
    constexpr int kBytes = static_cast<int>(sizeof(Shared<n>));
    auto* kern = space_kernel<decltype(t), n, WALK>;
    const cudaError_t err =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (err != cudaSuccess) return err;
    const int each = a.D / a.G, per = (each + Layout<n>::kChannels - 1) / Layout<n>::kChannels;
    kern<<<dim3(a.G * per, segments, a.B), kThreads, kBytes, stream>>>(a, sp);
    return cudaGetLastError();
  });
}

}  // namespace

cudaError_t launch_space_states(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                                cudaStream_t stream) {
  return launch<false>(a, sp, sp.segments - 1, f32, stream);
}
cudaError_t launch_space_walk(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                              cudaStream_t stream) {
  return launch<true>(a, sp, sp.segments, f32, stream);
}
cudaError_t launch_space_step(const SpaceArgs& a, bool f32, cudaStream_t stream) {
  const long long total = static_cast<long long>(a.B) * a.D * (a.N / 4);
  const long long grid = (total + kThreads - 1) / kThreads;
  if (grid > 2147483647LL) return cudaErrorInvalidValue;
  return by_states(a.N, f32, [&](auto t, auto n) {
    space_step_kernel<decltype(t), n>
        <<<static_cast<unsigned>(grid), kThreads, 0, stream>>>(a, total);
    return cudaGetLastError();
  });
}

}  // namespace gdr
