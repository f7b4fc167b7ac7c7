// Short causal convolution: one filter of K taps (2 to 4) for each channel,
//   s_t = bias + sum_{j<K} w[K-1-j] x_{t-j},   y = s sigmoid(s) or s,
// with taps that stop at a document's first token, and its gradients
//   ds = dy act'(s),  dx_t = sum_j w[K-1-j] ds_{t+j},  dw[K-1-j] = sum_t ds_t x_{t-j}.
//
// Streams: a thread walks a run of consecutive tokens of 4 channels with the last K - 1 inputs
// in registers, so that a token is read once per run plus K - 1 rows before it. What comes next
// is copied to the thread's own places in shared memory, two batches of 4 tokens ahead, which
// takes no registers and no barrier. Neighbouring threads have neighbouring channels.
// 65536 x 4096 bf16: 163 us, 0.97 of measured HBM bandwidth (two batches of 8 in registers:
// 176; 8 channels a thread, filter in single loads: 494). Gradients of 4 x 4096 x 4096: 86 us,
// 0.69 (batches in registers: 113; a branch for the activation at each token: 91); K = 2 takes 71,
// and 5 are the second launch.
#include <type_traits>

#include "column_sum.cuh"
#include "pair.cuh"
#include "short_conv.h"
#include "vec_io.cuh"

namespace gdr {
namespace {

// V elements as they are in memory (V = 4 or 8).
template <typename T, int V>
struct __align__(V * sizeof(T) > 16 ? 16 : V * sizeof(T)) Raw {
  static constexpr int kWords = V * sizeof(T) / 4;
  uint32_t u[kWords];
  // of 16 bytes or more, from rows that the kernel itself writes later
  __device__ __forceinline__ void load_written(const T* p) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p) + i);
      u[4 * i] = q.x;
      u[4 * i + 1] = q.y;
      u[4 * i + 2] = q.z;
      u[4 * i + 3] = q.w;
    }
  }
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
      u[0] = q.x;
      u[1] = q.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + i);
        u[4 * i] = q.x;
        u[4 * i + 1] = q.y;
        u[4 * i + 2] = q.z;
        u[4 * i + 3] = q.w;
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 2) {
      *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4*>(p)[i] =
            make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) u[i] = 0u;
  }
  __device__ __forceinline__ void get(float (&x)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) x[i] = __uint_as_float(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void get(f32x2 (&x)[V / 2]) const {
    float f[V];
    get(f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[i] = pair(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void put(const f32x2 (&x)[V / 2]) {
    float f[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) split(x[i], f[2 * i], f[2 * i + 1]);
    put(f);
  }
  __device__ __forceinline__ void put(const float (&x)[V]) {   // one rounding
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) u[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
      for (int i = 0; i < V / 2; ++i) u[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
  }
};

// The filter of V channels, as pairs of channels.
template <int K, int V>
__device__ __forceinline__ void load_filter(const ConvArgs& a, int c, f32x2 (&w)[K][V / 2],
                                            f32x2 (&bias)[V / 2]) {
  float f[V * K], g[V];     // V * K consecutive floats
  const float4* p = reinterpret_cast<const float4*>(a.weight + static_cast<long long>(c) * K);
#pragma unroll
  for (int i = 0; i < V * K / 4; ++i) {
    const float4 v = __ldg(p + i);
    f[4 * i] = v.x; f[4 * i + 1] = v.y; f[4 * i + 2] = v.z; f[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    const float4 v = a.bias ? __ldg(reinterpret_cast<const float4*>(a.bias + c) + i)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
    g[4 * i] = v.x; g[4 * i + 1] = v.y; g[4 * i + 2] = v.z; g[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][i] = pair(f[2 * i * K + k], f[(2 * i + 1) * K + k]);
    bias[i] = pair(g[2 * i], g[2 * i + 1]);
  }
}

// Row t of the sequence, t >= -(K - 1): the state's rows come before token 0.
template <typename T, int K, int V>
__device__ __forceinline__ void load_row(const ConvArgs& a, int b, int t, int c, Raw<T, V>& r) {
  if (t >= 0)
    r.load(static_cast<const T*>(a.x) + (static_cast<long long>(b) * a.T + t) * a.xs + c);
  else if (a.state)
    r.load(static_cast<const T*>(a.state) + (static_cast<long long>(b) * (K - 1) + K - 1 + t) * a.D + c);
  else
    r.zero();
}

// How many tokens behind token t are of its document, at most K - 1 (the state counts as
// the same one).
template <int K>
__device__ __forceinline__ int reach(const unsigned char* starts, int t) {
  int r = 0;
#pragma unroll
  for (int j = 0; j < K - 1; ++j)
    if (r == j && !(t - j >= 0 && starts[t - j])) r = j + 1;
  return r;
}

// The starts of four tokens, a byte each, of which `left` are there. As one word where they
// may be read so: nothing is done with it before it is needed (bytes put together at once
// cost the gradients 10% in waits for them).
__device__ __forceinline__ unsigned four_starts(const unsigned char* p, int left) {
  if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 3) == 0)
    return __ldg(reinterpret_cast<const unsigned*>(p));
  unsigned m = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (k < left) m |= static_cast<unsigned>(p[k]) << (8 * k);
  return m;
}

// A thread's V channels of a row, to shared memory.
template <typename T, int V>
__device__ __forceinline__ void copy_row(Raw<T, V>* to, const T* from) {
  constexpr int kBytes = V * static_cast<int>(sizeof(T));
  static_assert(kBytes == 8 || kBytes == 16, "");
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(to)), "l"(from), "n"(kBytes)
               : "memory");
}

constexpr int kFwdThreads = 128;
constexpr int kBatch = 4;          // tokens requested together
constexpr int kFwdStages = 3;      // batches on their way or in use (4: fp32 takes 198 us for 173)

template <typename T, int K>
__global__ void __launch_bounds__(kFwdThreads) short_conv_kernel(const ConvArgs a, int run,
                                                                 int runs, long long total) {
  constexpr int V = 4, H = V / 2;
  const long long id = static_cast<long long>(blockIdx.x) * kFwdThreads + threadIdx.x;
  if (id >= total) return;
  const int nv = a.D / V;
  const int c = static_cast<int>(id % nv) * V;
  const long long rest = id / nv;
  const int t0 = static_cast<int>(rest % runs) * run, b = static_cast<int>(rest / runs);
  const int t1 = min(t0 + run, a.T);
  const unsigned char* starts = a.starts ? a.starts + static_cast<long long>(b) * a.T : nullptr;
  const T* x = static_cast<const T*>(a.x) + static_cast<long long>(b) * a.T * a.xs + c;
  T* y = static_cast<T*>(a.y) + static_cast<long long>(b) * a.T * a.D + c;
  f32x2 w[K][H], bias[H], prev[K - 1][H];    // prev[j]: the row j + 1 tokens back
  __shared__ Raw<T, V> ring[kFwdStages][kBatch][kFwdThreads];
  unsigned marks[kFwdStages];                              // the batches' documents' starts
  const T* xp = x + static_cast<long long>(t0) * a.xs;     // the next batch's
  auto fetch = [&](int stage, int t) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k, xp += a.xs)
      if (t + k < t1) copy_row(&ring[stage][k][threadIdx.x], xp);
    asm volatile("cp.async.commit_group;" ::: "memory");
    marks[stage] = starts && t < t1 ? four_starts(starts + t, t1 - t) : 0;
  };
#pragma unroll
  for (int i = 0; i < kFwdStages - 1; ++i) fetch(i, t0 + i * kBatch);
  load_filter<K, V>(a, c, w, bias);
  {
    Raw<T, V> r[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) load_row<T, K, V>(a, b, t0 - 1 - j, c, r[j]);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) r[j].get(prev[j]);
  }
  if (starts && t0 > 0) {      // the run's first token may be in the middle of a document
    const int r = reach<K>(starts, t0 - 1);
#pragma unroll
    for (int j = 1; j < K - 1; ++j)
      if (j > r)
#pragma unroll
        for (int i = 0; i < H; ++i) prev[j][i] = 0;
  }
  T* yp = y + static_cast<long long>(t0) * a.D;
  auto token = [&](const Raw<T, V>& raw, auto activated) {
    f32x2 v[H], s[H];
    raw.get(v);
#pragma unroll
    for (int i = 0; i < H; ++i) {
      s[i] = fma2(w[K - 1][i], v[i], bias[i]);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) s[i] = fma2(w[K - 2 - j][i], prev[j][i], s[i]);
      if (decltype(activated)::value) s[i] = mul2(s[i], sigmoid2(s[i]));
    }
    Raw<T, V> out;
    out.put(s);
    out.store(yp);
    yp += a.D;
#pragma unroll
    for (int j = K - 2; j > 0; --j)
#pragma unroll
      for (int i = 0; i < H; ++i) prev[j][i] = prev[j - 1][i];
#pragma unroll
    for (int i = 0; i < H; ++i) prev[0][i] = v[i];
  };
  auto tokens = [&](int stage, int t, auto activated) {
    if (t + kBatch <= t1 && marks[stage] == 0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) token(ring[stage][k][threadIdx.x], activated);
    } else {
#pragma unroll 1
      for (int k = 0; k < kBatch && t + k < t1; ++k) {
        if ((marks[stage] >> (8 * k)) & 0xff)
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int i = 0; i < H; ++i) prev[j][i] = 0;
        token(ring[stage][k][threadIdx.x], activated);
      }
    }
  };
  auto walk = [&](auto activated) {
    for (int t = t0; t < t1; t += kFwdStages * kBatch) {
#pragma unroll
      for (int i = 0; i < kFwdStages; ++i) {
        fetch((i + kFwdStages - 1) % kFwdStages, t + (i + kFwdStages - 1) * kBatch);
        asm volatile("cp.async.wait_group %0;" ::"n"(kFwdStages - 1) : "memory");
        tokens(i, t + i * kBatch, activated);
      }
    }
  };
  if (a.silu)
    walk(std::true_type{});
  else
    walk(std::false_type{});
  if (t1 == a.T && a.state_out) {     // prev is the last rows, zeros behind a start
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
      Raw<T, V> r;
      r.put(prev[j]);
      r.store(static_cast<T*>(a.state_out) +
              (static_cast<long long>(b) * (K - 1) + K - 2 - j) * a.D + c);
    }
  }
}

// Gradients: a warp has 128 channels (4 a thread) of one run of tokens, a CTA kRuns
// neighbouring runs, whose filter gradients it adds up in a fixed order to one row of
// `partial` ([K + 1, D], the last row the bias's); column_sum adds those rows. A run walks
// K - 1 tokens past its end for what they pass back.
constexpr int kRuns = 4;
constexpr int kBwdThreads = 32 * kRuns;
constexpr int kBwdBatch = 4;
// CTAs of an SM, which registers bound
constexpr int bwd_ctas(int K, bool f32) { return f32 && K > 2 ? 3 : 4; }
constexpr int kStages = 3;         // batches on their way or in use (6 leave fewer CTAs: 159 us)

template <typename T, int K>
__global__ void __launch_bounds__(kBwdThreads, bwd_ctas(K, sizeof(T) == 4))
    short_conv_bwd_kernel(const ConvArgs a, int run, int groups, int slices) {
  constexpr int V = 4, H = V / 2;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  Raw<T, V>* ring = reinterpret_cast<Raw<T, V>*>(raw_smem);   // [kStages][kBwdBatch][2][threads]
  __shared__ __align__(16) float sums[kRuns][K + 1][32 * V];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int slice = blockIdx.x % slices, c = (slice * 32 + lane) * V;
  const int rest = blockIdx.x / slices, b = rest / groups, group = rest % groups;
  const int t0 = (group * kRuns + warp) * run, t1 = min(t0 + run, a.T);
  f32x2 dw[K + 1][H];
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int i = 0; i < H; ++i) dw[k][i] = 0;
  if (c < a.D && t0 < a.T) {
    const unsigned char* starts = a.starts ? a.starts + static_cast<long long>(b) * a.T : nullptr;
    const T* xp = static_cast<const T*>(a.x) + static_cast<long long>(b) * a.T * a.xs + c;
    const T* dyp = static_cast<const T*>(a.dy) + static_cast<long long>(b) * a.T * a.D + c;
    T* dxp = static_cast<T*>(a.dx) + static_cast<long long>(b) * a.T * a.D + c;
    T* dst = a.dstate ? static_cast<T*>(a.dstate) + static_cast<long long>(b) * (K - 1) * a.D + c
                      : nullptr;
    const int stop = min(t1 + K - 1, a.T);
    f32x2 w[K][H], bias[H], prev[K - 1][H], acc[K][H];   // acc[j]: dx of the token j back (j > 0)
    const T* xf = xp + static_cast<long long>(t0) * a.xs;     // the next batch's
    const T* yf = dyp + static_cast<long long>(t0) * a.D;
    unsigned marks[kStages];          // the batches' documents' starts
    auto place = [&](int stage, int k, int which) {
      return ring + ((stage * kBwdBatch + k) * 2 + which) * kBwdThreads + threadIdx.x;
    };
    auto fetch = [&](int stage, int t) {
#pragma unroll
      for (int k = 0; k < kBwdBatch; ++k, xf += a.xs, yf += a.D)
        if (t + k < stop) {
          copy_row(place(stage, k, 0), xf);
          copy_row(place(stage, k, 1), yf);
        }
      asm volatile("cp.async.commit_group;" ::: "memory");
      marks[stage] = starts ? four_starts(starts + t, stop - t) : 0;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i, t0 + i * kBwdBatch);
    load_filter<K, V>(a, c, w, bias);
    {
      Raw<T, V> r[K - 1];
#pragma unroll
      for (int j = 0; j < K - 1; ++j) load_row<T, K, V>(a, b, t0 - 1 - j, c, r[j]);
#pragma unroll
      for (int j = 0; j < K - 1; ++j) r[j].get(prev[j]);
    }
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int i = 0; i < H; ++i) acc[j][i] = 0;
    // tokens behind the current one that are of its document, up to K - 1
    int back = K - 2;
    if (starts && t0 > 0) back = reach<K>(starts, t0 - 1);
    // rows of dx are finished K - 1 tokens later; where the current token's goes
    T* dxo = dxp + (static_cast<long long>(t0) - (K - 1)) * a.D;
    // a finished row: of this run's tokens, or the state's before the first
    auto emit = [&](int e, const f32x2 (&v)[H]) {
      Raw<T, V> r;
      r.put(v);
      if (e >= t0)
        r.store(dxp + static_cast<long long>(e) * a.D);
      else if (t0 == 0 && dst)
        r.store(dst + static_cast<long long>(K - 1 + e) * a.D);
    };
    // one token; INNER: of the run, with K - 1 others of its document and the run behind it
    auto token = [&](const Raw<T, V>& raw_x, const Raw<T, V>& raw_y, int now, auto inner, auto activated) {
      constexpr bool INNER = decltype(inner)::value, SILU = decltype(activated)::value;
      f32x2 v[H], g[H];
      raw_x.get(v);
      raw_y.get(g);
      if (!INNER && back < K - 1)
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
          if (j + 1 > back)
#pragma unroll
            for (int i = 0; i < H; ++i) prev[j][i] = 0;
#pragma unroll
      for (int i = 0; i < H; ++i) {
        if (SILU) {
          f32x2 s = fma2(w[K - 1][i], v[i], bias[i]);
#pragma unroll
          for (int j = 0; j < K - 1; ++j) s = fma2(w[K - 2 - j][i], prev[j][i], s);
          // sg (1 + s (1 - sg)) = sg + (s sg) (1 - sg)
          const f32x2 sg = sigmoid2(s), one = both(1.f);
          const f32x2 slope = fma2(mul2(s, sg), fma2(sg, both(-1.f), one), sg);
          g[i] = mul2(g[i], slope);
        }
      }
#pragma unroll
      for (int j = 1; j < K; ++j)
        if (INNER || j <= back)
#pragma unroll
          for (int i = 0; i < H; ++i) acc[j][i] = fma2(w[K - 1 - j][i], g[i], acc[j][i]);
      if (INNER || now < t1)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          dw[K - 1][i] = fma2(g[i], v[i], dw[K - 1][i]);
#pragma unroll
          for (int j = 0; j < K - 1; ++j)
            dw[K - 2 - j][i] = fma2(g[i], prev[j][i], dw[K - 2 - j][i]);
          dw[K][i] = add2(dw[K][i], g[i]);
        }
      if (INNER) {
        Raw<T, V> r;
        r.put(acc[K - 1]);
        r.store(dxo);
      } else {
        emit(now - (K - 1), acc[K - 1]);
      }
      dxo += a.D;
#pragma unroll
      for (int j = K - 1; j > 1; --j)
#pragma unroll
        for (int i = 0; i < H; ++i) acc[j][i] = acc[j - 1][i];
#pragma unroll
      for (int i = 0; i < H; ++i) acc[1][i] = mul2(w[K - 1][i], g[i]);
#pragma unroll
      for (int j = K - 2; j > 0; --j)
#pragma unroll
        for (int i = 0; i < H; ++i) prev[j][i] = prev[j - 1][i];
#pragma unroll
      for (int i = 0; i < H; ++i) prev[0][i] = v[i];
    };
    auto tokens = [&](int stage, int t, auto activated) {
      auto load = [&](int k, int which) { return *place(stage, k, which); };
      if (marks[stage] == 0 && back == K - 1 && t - (K - 1) >= t0 && t + kBwdBatch <= t1) {
#pragma unroll
        for (int k = 0; k < kBwdBatch; ++k) token(load(k, 0), load(k, 1), t + k, std::true_type{}, activated);
      } else {
#pragma unroll 1
        for (int k = 0; k < kBwdBatch && t + k < stop; ++k) {
          back = (marks[stage] >> (8 * k)) & 0xff ? 0 : min(back + 1, K - 1);
          token(load(k, 0), load(k, 1), t + k, std::false_type{}, activated);
        }
      }
    };
    auto walk = [&](auto activated) {
      for (int t = t0; t < stop; t += kStages * kBwdBatch) {
#pragma unroll
        for (int i = 0; i < kStages; ++i) {
          fetch((i + kStages - 1) % kStages, t + (i + kStages - 1) * kBwdBatch);
          asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
          tokens(i, t + i * kBwdBatch, activated);
        }
      }
    };
    if (a.silu)
      walk(std::true_type{});
    else
      walk(std::false_type{});
    if (stop == a.T) {   // what is behind the last token comes from the state's gradient
#pragma unroll
      for (int j = 1; j < K; ++j) {
        const int e = a.T - j;
        if (a.dstate_out && j - 1 <= back) {
          Raw<T, V> r;
          f32x2 g[H];
          r.load(static_cast<const T*>(a.dstate_out) +
                 (static_cast<long long>(b) * (K - 1) + K - 1 - j) * a.D + c);
          r.get(g);
#pragma unroll
          for (int i = 0; i < H; ++i) acc[j][i] = add2(acc[j][i], g[i]);
        }
        if (e < t1) emit(e, acc[j]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k <= K; ++k) {
    float f[V];
#pragma unroll
    for (int i = 0; i < H; ++i) split(dw[k][i], f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<float4*>(&sums[warp][k][lane * V]) = make_float4(f[0], f[1], f[2], f[3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < (K + 1) * 32 * V; i += kBwdThreads) {
    const int k = i / (32 * V), j = i % (32 * V), d = slice * 32 * V + j;
    float s = sums[0][k][j];
#pragma unroll
    for (int r = 1; r < kRuns; ++r) s += sums[r][k][j];
    if (d < a.D) a.partial[(static_cast<size_t>(rest) * (K + 1) + k) * a.D + d] = s;
  }
}

__global__ void __launch_bounds__(256) filter_grad_kernel(const ConvArgs a, int rows) {
  column_sum<8>(a.partial, rows, (a.K + 1) * a.D, [&](int i, float s) {
    const int k = i / a.D, d = i % a.D;
    if (k < a.K)
      a.dweight[static_cast<long long>(d) * a.K + k] = s;
    else if (a.dbias)
      a.dbias[d] = s;
  });
}

// One token of each sequence: a thread has 8 channels of R sequences, for which it reads the
// filter (more bytes than a sequence's rows) once.
template <typename T, int K, int R>
__global__ void __launch_bounds__(kFwdThreads) short_conv_step_kernel(const ConvArgs a,
                                                                      long long total) {
  constexpr int V = 8;
  const long long id = static_cast<long long>(blockIdx.x) * kFwdThreads + threadIdx.x;
  if (id >= total) return;
  const int nv = a.D / V, c = static_cast<int>(id % nv) * V;
  const long long b0 = id / nv * R;
  T* st = static_cast<T*>(a.state_out) + b0 * (K - 1) * a.D + c;
  Raw<T, V> r[R][K];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (b0 + i >= a.B) break;
#pragma unroll
    for (int k = 0; k < K - 1; ++k)
      r[i][k].load_written(st + (i * (K - 1) + k) * static_cast<long long>(a.D));
    r[i][K - 1].load(static_cast<const T*>(a.x) + (b0 + i) * a.xs + c);
  }
  f32x2 w[K][V / 2], bias[V / 2];
  load_filter<K, V>(a, c, w, bias);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (b0 + i >= a.B) break;
    f32x2 s[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) s[j] = bias[j];
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      f32x2 v[V / 2];
      r[i][k].get(v);
#pragma unroll
      for (int j = 0; j < V / 2; ++j) s[j] = fma2(w[k][j], v[j], s[j]);
    }
    if (a.silu)
#pragma unroll
      for (int j = 0; j < V / 2; ++j) s[j] = mul2(s[j], sigmoid2(s[j]));
    Raw<T, V> out;
    out.put(s);
    out.store(static_cast<T*>(a.y) + (b0 + i) * a.D + c);
#pragma unroll
    for (int k = 0; k < K - 1; ++k) r[i][k + 1].store(st + (i * (K - 1) + k) * static_cast<long long>(a.D));
  }
}

template <class F>
cudaError_t by_taps(int K, bool f32, F f) {
  using std::integral_constant;
  auto typed = [&](auto k) { return f32 ? f(float{}, k) : f(__nv_bfloat16{}, k); };
  if (K == 2) return typed(integral_constant<int, 2>{});
  if (K == 3) return typed(integral_constant<int, 3>{});
  return typed(integral_constant<int, 4>{});
}

// Tokens of a run of the backward, and the CTAs' rows of partial sums, one for each batch row
// and kRuns runs. The run is what takes least time by waves of four CTAs an SM, a run being
// K - 1 tokens and its start, about 6 in all, longer than its own (4 x 4096 x 4096 bf16: 91 us
// with runs of 116 in 1.9 waves, 95 with 120 or 64, 100 with 48, 103 with 32).
int bwd_groups(int T, int run) { return (T + kRuns * run - 1) / (kRuns * run); }
int bwd_run(int B, int T, int D, int K, bool f32) {
  const int ctas = bwd_ctas(K, f32) * 152;
  const long long slices = static_cast<long long>((D + 127) / 128) * B;
  int best = 128;                       // multiples of 4: see four_starts
  long long least = 0;
  for (int run = 128; run >= 8; run -= 4) {
    const long long waves = (slices * bwd_groups(T, run) + ctas - 1) / ctas;
    const long long cost = waves * (run + 6);
    if (run == 128 || cost < least) {
      least = cost;
      best = run;
    }
  }
  return best;
}

}  // namespace

size_t short_conv_bwd_workspace_bytes(int B, int T, int D, int K, bool f32) {
  return static_cast<size_t>(B) * bwd_groups(T, bwd_run(B, T, D, K, f32)) * (K + 1) * D *
         sizeof(float);
}

cudaError_t launch_short_conv(const ConvArgs& a, bool f32, cudaStream_t stream) {
  // long runs where those fill the GPU's threads, else short ones
  const long long vecs = static_cast<long long>(a.B) * (a.D / 4);
  int run = 64;
  while (run > 8 && vecs * ((a.T + run - 1) / run) < 152 * 2048) run /= 2;
  const int runs = (a.T + run - 1) / run;
  const long long total = vecs * runs, grid = (total + kFwdThreads - 1) / kFwdThreads;
  if (grid > 2147483647LL) return cudaErrorInvalidValue;
  return by_taps(a.K, f32, [&](auto t, auto k) {
    short_conv_kernel<decltype(t), k><<<static_cast<unsigned>(grid), kFwdThreads, 0, stream>>>(
        a, run, runs, total);
    return cudaGetLastError();
  });
}

cudaError_t launch_short_conv_bwd(const ConvArgs& a, bool f32, cudaStream_t stream) {
  const int run = bwd_run(a.B, a.T, a.D, a.K, f32), groups = bwd_groups(a.T, run);
  const int slices = (a.D + 127) / 128;
  const long long grid = static_cast<long long>(slices) * a.B * groups;
  if (grid > 2147483647LL) return cudaErrorInvalidValue;
  return by_taps(a.K, f32, [&](auto t, auto k) {
    constexpr int kBytes = kStages * kBwdBatch * 2 * kBwdThreads * 4 * sizeof(decltype(t));
    const cudaError_t err = cudaFuncSetAttribute(
        short_conv_bwd_kernel<decltype(t), k>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (err != cudaSuccess) return err;
    short_conv_bwd_kernel<decltype(t), k>
        <<<static_cast<unsigned>(grid), kBwdThreads, kBytes, stream>>>(a, run, groups, slices);
    filter_grad_kernel<<<((a.K + 1) * a.D + 31) / 32, 256, 0, stream>>>(a, a.B * groups);
    return cudaGetLastError();
  });
}

cudaError_t launch_short_conv_step(const ConvArgs& a, bool f32, cudaStream_t stream) {
  auto run = [&](auto rows) {
    constexpr int R = decltype(rows)::value;
    const long long total = (static_cast<long long>(a.B) + R - 1) / R * (a.D / 8);
    const long long grid = (total + kFwdThreads - 1) / kFwdThreads;
    if (grid > 2147483647LL) return cudaErrorInvalidValue;
    return by_taps(a.K, f32, [&](auto t, auto k) {
      short_conv_step_kernel<decltype(t), k, R>
          <<<static_cast<unsigned>(grid), kFwdThreads, 0, stream>>>(a, total);
      return cudaGetLastError();
    });
  };
  // two sequences a thread where that leaves two CTAs for each SM
  if (static_cast<long long>(a.B) * (a.D / 8) >= 4 * 152 * kFwdThreads)
    return run(std::integral_constant<int, 2>{});
  return run(std::integral_constant<int, 1>{});
}

}  // namespace gdr
