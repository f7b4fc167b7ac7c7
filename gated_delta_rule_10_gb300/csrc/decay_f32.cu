// Linear attention with a decay for each head, chunked, for fp32 inputs.
//
// With G the in-chunk running sum of the log-decay (inclusive) and chunks of
// C = 64 tokens,
//   o_r     = s (e^{G_r} S_n^T q_r + sum_{i<=r} e^{G_r-G_i} (q_r . k_i) v_i)
//   S_{n+1} = e^{G_C} S_n + sum_i e^{G_C-G_i} k_i v_i^T
// and, with D the gradient of S and dO that of o,
//   dq_r = s (e^{G_r} S_n dO_r + sum_{i<=r} e^{G_r-G_i} (dO_r . v_i) k_i)
//   dv_i = s sum_{r>=i} e^{G_r-G_i} (q_r . k_i) dO_r + e^{G_C-G_i} D_{n+1}^T k_i
//   dk_i = s sum_{r>=i} e^{G_r-G_i} (dO_r . v_i) q_r + e^{G_C-G_i} D_{n+1} v_i
//   D_n  = e^{G_C} D_{n+1} + s sum_r e^{G_r} q_r dO_r^T.
// The gate's gradient takes, with M_ri = s e^{G_r-G_i} (q_r . k_i)(dO_r . v_i) over
// the pairs i < r, from every token (gate_grad_kernel joins them)
//   what comes from before its block of 32: s e^{G_t} q_t . (S_n dO_t) + sum of M_ti
//   what goes to after it: e^{G_C-G_t} k_t . (D_{n+1} v_t) + sum of M_rt
//   and within the block the difference of its row's and its column's sums.
// dq walks the chunks forward with S, dk and dv walk them backward with D; the
// two walks are independent and run as two halves of one grid.
//
// Every product runs on the warp-level tensor cores with each fp32 operand split
// into tf32 hi + lo (three products, about 2^-21 relative), which keeps fp32
// results fp32. One CTA owns a (batch, head, segment of the sequence) with its
// state in shared memory; the tiles are fp32 with rows padded by 4 floats.
// Bound by the warp products: every operand is read from shared memory and split where
// it is used, ~10 us a chunk of 64 at 128 x 128 (4 x 2048 x 16 x 128: forward 600 us,
// backward 1.8 ms; 1 x 257 x 2 x 64: 31 us, launches and one chunk).
#include "common.cuh"
#include "decay.h"

namespace gdr {
namespace {

constexpr int kC = 64;
constexpr int kThreads = 256;

__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(hi) : "f"(x));
  const float r = x - __uint_as_float(hi);
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(lo) : "f"(r));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A shared-memory fp32 matrix seen through two strides (a transpose is a swap).
struct View {
  const float* p;
  int row, col;
  __device__ __forceinline__ float at(int r, int c) const { return p[r * row + c * col]; }
};

// One warp's part of an M x N product over K: the eight warps sit 4 x 2, each
// with MT x NT tiles of 16 x 8.
template <int M, int N>
struct Acc {
  static constexpr int MT = M / 64, NT = N / 16;
  float v[MT][NT][4];
  __device__ __forceinline__ static int row0(int mt) {
    return (threadIdx.x >> 6) * (M / 4) + mt * 16 + ((threadIdx.x & 31) >> 2);
  }
  __device__ __forceinline__ static int col0(int nt) {
    return ((threadIdx.x >> 5) & 1) * (N / 2) + nt * 8 + 2 * (threadIdx.x & 3);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[m][n][i] = 0.f;
  }
  // f(row, col, value) for every element of this thread; value by reference
  template <class F>
  __device__ __forceinline__ void each(F f) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f(row0(m) + (i >> 1) * 8, col0(n) + (i & 1), v[m][n][i]);
  }
  // v += A (M x K) B (K x N)
  template <int K>
  __device__ __forceinline__ void mul(View A, View B) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int r0 = (threadIdx.x >> 6) * (M / 4), c0 = ((threadIdx.x >> 5) & 1) * (N / 2);
#pragma unroll 2
    for (int k = 0; k < K; k += 8) {
      uint32_t ah[MT][4], al[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          split_tf32(A.at(r0 + m * 16 + g + (i & 1) * 8, k + t + (i >> 1) * 4), ah[m][i], al[m][i]);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint32_t bh[2], bl[2];
        split_tf32(B.at(k + t, c0 + n * 8 + g), bh[0], bl[0]);
        split_tf32(B.at(k + t + 4, c0 + n * 8 + g), bh[1], bl[1]);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          // the tensor cores truncate as they add: each step's products are added up
          // by themselves, and to the sum with rounding
          float p[4] = {0.f, 0.f, 0.f, 0.f};
          mma_tf32(p, al[m], bh[0], bh[1]);
          mma_tf32(p, ah[m], bl[0], bl[1]);
          mma_tf32(p, ah[m], bh[0], bh[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[m][n][i] += p[i];
        }
      }
    }
  }
};

// The chunk's decay factors. The running sums are taken in fp64 and kept as
// hi + lo pairs, so that a difference of two of them is exact to fp32 whatever
// their size; a clearing token (kDecayReset) leaves the sums and cuts by index.
struct Gates {
  float hi[kC], lo[kC];   // G
  float head[kC];         // e^{G_r}, 0 once a token of the chunk has cleared the state
  float tail[kC];         // e^{G_C - G_i}, 0 if a later token clears
  int cut[kC];            // last clearing token at or before r, -1: none
  float sum;              // G_C, minus infinity if a token clears
  __device__ __forceinline__ float between(int r, int i) const {
    return i <= r && i >= cut[r] ? expf((hi[r] - hi[i]) + (lo[r] - lo[i])) : 0.f;
  }
};

// One warp fills the gates of the chunk's `n` tokens (the rest have decay 1).
__device__ void load_gates(Gates& s, const DecayArgs& a, int b, int h, int t0, int n) {
  const int lane = threadIdx.x & 31;
  double x[2];
  int c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * lane + i;
    float g = 0.f;
    if (r < n)
      g = a.per_head ? a.g[h] : a.g[(static_cast<size_t>(b) * a.T + t0 + r) * a.H + h];
    const bool clear = g <= kDecayReset;
    x[i] = clear ? 0.0 : static_cast<double>(g);
    c[i] = clear ? r : -1;
  }
  x[1] += x[0];
  c[1] = max(c[0], c[1]);
  double sum = x[1];
  int last = c[1];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double y = __shfl_up_sync(0xffffffffu, sum, off);
    const int z = __shfl_up_sync(0xffffffffu, last, off);
    if (lane >= off) {
      sum += y;
      last = max(last, z);
    }
  }
  double before = __shfl_up_sync(0xffffffffu, sum, 1);
  int lb = __shfl_up_sync(0xffffffffu, last, 1);
  if (lane == 0) {
    before = 0.0;
    lb = -1;
  }
  const double total = __shfl_sync(0xffffffffu, sum, 31);
  const int lt = __shfl_sync(0xffffffffu, last, 31);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 2 * lane + i;
    const double G = before + x[i];
    const int cut = max(lb, c[i]);
    s.hi[r] = static_cast<float>(G);
    s.lo[r] = static_cast<float>(G - static_cast<double>(s.hi[r]));
    s.cut[r] = cut;
    s.head[r] = cut < 0 ? expf(static_cast<float>(G)) : 0.f;
    s.tail[r] = lt <= r ? expf(static_cast<float>(total - G)) : 0.f;
  }
  if (lane == 0) s.sum = lt < 0 ? static_cast<float>(total) : -INFINITY;
}

// Rows [t0, t0 + n) of one head into a 64 x W tile, zeros past n.
template <int W>
__device__ void load_tile(float* dst, const float* src, long long stride, int n) {
  constexpr int V = W / 8, LD = W + 4;
  for (int i = threadIdx.x; i < kC * V; i += kThreads) {
    const int r = i / V, c = i % V;
    float x[8] = {};
    if (r < n) load8(src + r * stride + 8 * c, x);
    float4* d = reinterpret_cast<float4*>(dst + r * LD + 8 * c);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

struct Where {
  int b, h, bh, t0, t1;
  size_t tok;   // b * T
};
__device__ __forceinline__ Where where(const DecayArgs& a, int len, int seg) {
  Where w;
  w.bh = blockIdx.y;
  w.b = w.bh / a.H;
  w.h = w.bh % a.H;
  w.t0 = seg * len;
  w.t1 = min(a.T, w.t0 + len);
  w.tok = static_cast<size_t>(w.b) * a.T;
  return w;
}
__device__ __forceinline__ const float* rows_of(const void* p, const Where& w, int t,
                                            long long stride, int head_off) {
  return static_cast<const float*>(p) + static_cast<long long>(w.tok + t) * stride + head_off;
}

template <int NK, int NV>
__device__ void load_state(float* S, const float* src) {
  for (int i = threadIdx.x; i < NK * NV; i += kThreads)
    S[(i / NV) * (NV + 4) + i % NV] = src ? src[i] : 0.f;
}
template <int NK, int NV>
__device__ void store_state(const float* S, float* dst) {
  for (int i = threadIdx.x; i < NK * NV; i += kThreads)
    dst[i] = S[(i / NV) * (NV + 4) + i % NV];
}

// S = e^sum S + X^T Y over the chunk's tokens (X: 64 x NK, Y: 64 x NV, one of
// them scaled by the caller)
template <int NK, int NV>
__device__ __forceinline__ void update_state(float* S, float sum, const float* X, const float* Y) {
  Acc<NK, NV> acc;
  const float d = decay_code(sum);
  acc.each([&](int r, int c, float& x) { x = decayed(d, S[r * (NV + 4) + c], 0.f); });
  acc.template mul<kC>(View{X, 1, NK + 4}, View{Y, NV + 4, 1});
  acc.each([&](int r, int c, float& x) { S[r * (NV + 4) + c] = x; });
}
template <int W>
__device__ __forceinline__ void scale_rows(float* X, const float* f) {
  for (int i = threadIdx.x; i < kC * W; i += kThreads) X[(i / W) * (W + 4) + i % W] *= f[i / W];
}

// Local end state of every piece from a zero state (REV: the gradient of its
// start state from a zero gradient at its end), and its decay.
template <int NK, int NV, bool REV>
__global__ void __launch_bounds__(kThreads, 1) states_f32(const DecayArgs a, const DecaySplit sp) {
  extern __shared__ __align__(16) float sm[];
  float *S = sm, *X = S + NK * (NV + 4), *Y = X + kC * (NK + 4);
  __shared__ Gates gates;
  const int seg = static_cast<int>(blockIdx.x) + (REV ? sp.slot_of(1) : 0);   // (no D before)
  const Where w = where(a, sp.piece_len, seg);
  const int hk = w.h / (a.H / a.Hk);
  load_state<NK, NV>(S, nullptr);
  float sum = 0.f;
  const int chunks = (w.t1 - w.t0 + kC - 1) / kC;
  for (int i = 0; i < chunks; ++i) {
    const int t = w.t0 + (REV ? chunks - 1 - i : i) * kC, n = min(kC, w.t1 - t);
    __syncthreads();
    if (threadIdx.x < 32) load_gates(gates, a, w.b, w.h, t, n);
    if (REV) {
      load_tile<NK>(X, rows_of(a.q, w, t, a.sq, hk * NK), a.sq, n);
      load_tile<NV>(Y, rows_of(a.dO, w, t, static_cast<long long>(a.H) * NV, w.h * NV),
                    static_cast<long long>(a.H) * NV, n);
    } else {
      load_tile<NK>(X, rows_of(a.k, w, t, a.sk, hk * NK), a.sk, n);
      load_tile<NV>(Y, rows_of(a.v, w, t, a.sv, w.h * NV), a.sv, n);
    }
    __syncthreads();
    scale_rows<NV>(Y, REV ? gates.head : gates.tail);
    __syncthreads();
    update_state<NK, NV>(S, gates.sum, X, Y);
    sum += gates.sum;
  }
  __syncthreads();
  const int slot = REV ? seg : seg + 1;
  float* dst = (REV ? sp.D : sp.S) + (static_cast<size_t>(w.bh) * sp.slots + slot) * NK * NV;
  if (REV)
    for (int i = threadIdx.x; i < NK * NV; i += kThreads)
      dst[i] = a.scale * S[(i / NV) * (NV + 4) + i % NV];
  else
    store_state<NK, NV>(S, dst);
  if (threadIdx.x == 0) sp.decay[static_cast<size_t>(w.bh) * sp.pieces + seg] = decay_code(sum);
}

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads, 1) fwd_f32(const DecayArgs a, const DecaySplit sp) {
  extern __shared__ __align__(16) float sm[];
  float *S = sm, *Q = S + NK * (NV + 4), *K = Q + kC * (NK + 4), *V = K + kC * (NK + 4),
        *A = V + kC * (NV + 4);
  __shared__ Gates gates;
  const Where w = where(a, sp.seg_len, blockIdx.x);
  const int hk = w.h / (a.H / a.Hk);
  const float* start = sp.segments > 1
                           ? sp.S + (static_cast<size_t>(w.bh) * sp.slots + sp.slot_of(blockIdx.x)) * NK * NV
                           : (a.h0 ? a.h0 + static_cast<size_t>(w.bh) * NK * NV : nullptr);
  load_state<NK, NV>(S, start);
  for (int t = w.t0; t < w.t1; t += kC) {
    const int n = min(kC, w.t1 - t);
    __syncthreads();
    if (threadIdx.x < 32) load_gates(gates, a, w.b, w.h, t, n);
    load_tile<NK>(Q, rows_of(a.q, w, t, a.sq, hk * NK), a.sq, n);
    load_tile<NK>(K, rows_of(a.k, w, t, a.sk, hk * NK), a.sk, n);
    load_tile<NV>(V, rows_of(a.v, w, t, a.sv, w.h * NV), a.sv, n);
    __syncthreads();
    {
      Acc<kC, kC> s;
      s.zero();
      s.template mul<NK>(View{Q, NK + 4, 1}, View{K, 1, NK + 4});
      s.each([&](int r, int c, float& x) { A[r * (kC + 4) + c] = x * gates.between(r, c); });
    }
    Acc<kC, NV> o;
    o.zero();
    o.template mul<NK>(View{Q, NK + 4, 1}, View{S, NV + 4, 1});
    o.each([&](int r, int, float& x) { x *= gates.head[r]; });
    __syncthreads();
    o.template mul<kC>(View{A, kC + 4, 1}, View{V, NV + 4, 1});
    float* out = static_cast<float*>(a.o);
    o.each([&](int r, int c, float& x) {
      if (r < n) out[((w.tok + t + r) * a.H + w.h) * NV + c] = a.scale * x;
    });
    __syncthreads();
    scale_rows<NV>(V, gates.tail);
    __syncthreads();
    update_state<NK, NV>(S, gates.sum, K, V);
  }
  __syncthreads();
  if (a.hT && blockIdx.x == gridDim.x - 1)
    store_state<NK, NV>(S, a.hT + static_cast<size_t>(w.bh) * NK * NV);
}

// blockIdx.z = 0: dq and the states' part of what comes from before, forward with
// S. 1: dk, dv and the other terms, backward with D.
template <int NK, int NV>
__global__ void __launch_bounds__(kThreads, 1) bwd_f32(const DecayArgs a, const DecaySplit sp) {
  extern __shared__ __align__(16) float sm[];
  float *S = sm, *Q = S + NK * (NV + 4), *K = Q + kC * (NK + 4), *V = K + kC * (NK + 4),
        *O = V + kC * (NV + 4), *A = O + kC * (NV + 4);
  __shared__ Gates gates;
  __shared__ float flow[6][kC];
  const Where w = where(a, sp.seg_len, blockIdx.x);
  const int hk = w.h / (a.H / a.Hk);
  const bool rev = blockIdx.z == 1;
  const size_t st = static_cast<size_t>(NK) * NV;
  const float* start;
  if (!rev)
    start = sp.segments > 1 ? sp.S + (static_cast<size_t>(w.bh) * sp.slots + sp.slot_of(blockIdx.x)) * st
                            : (a.h0 ? a.h0 + w.bh * st : nullptr);
  else
    start = sp.segments > 1 ? sp.D + (static_cast<size_t>(w.bh) * sp.slots + sp.slot_of(blockIdx.x + 1)) * st
                            : (a.dhT ? a.dhT + w.bh * st : nullptr);
  load_state<NK, NV>(S, start);
  const long long so = static_cast<long long>(a.H) * NV;
  const int chunks = (w.t1 - w.t0 + kC - 1) / kC;
  float* dq = static_cast<float*>(a.dq);
  float* dk = static_cast<float*>(a.dk);
  float* dv = static_cast<float*>(a.dv);
  const int wn = (threadIdx.x >> 5) & 1, lane = threadIdx.x & 31;
  for (int i = 0; i < chunks; ++i) {
    const int t = w.t0 + (rev ? chunks - 1 - i : i) * kC, n = min(kC, w.t1 - t);
    __syncthreads();
    if (threadIdx.x < 32) load_gates(gates, a, w.b, w.h, t, n);
    for (int j = threadIdx.x; j < 6 * kC; j += kThreads) flow[j / kC][j % kC] = 0.f;
    load_tile<NK>(Q, rows_of(a.q, w, t, a.sq, hk * NK), a.sq, n);
    load_tile<NK>(K, rows_of(a.k, w, t, a.sk, hk * NK), a.sk, n);
    load_tile<NV>(V, rows_of(a.v, w, t, a.sv, w.h * NV), a.sv, n);
    load_tile<NV>(O, rows_of(a.dO, w, t, so, w.h * NV), so, n);
    __syncthreads();
    Acc<kC, kC> dA;
    dA.zero();
    dA.template mul<NV>(View{O, NV + 4, 1}, View{V, 1, NV + 4});
    // a thread's part of each of its two rows, summed over the four lanes that
    // share them and added by the two column halves in a fixed order
    auto row_flow = [&](auto& acc, const float* X, float* out) {
      float part[2] = {0.f, 0.f};
      acc.each([&](int r, int c, float& x) { part[(r >> 3) & 1] += x * X[r * (NK + 4) + c]; });
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        part[p] += __shfl_xor_sync(0xffffffffu, part[p], 1);
        part[p] += __shfl_xor_sync(0xffffffffu, part[p], 2);
        if ((lane & 3) == 0) out[wn * kC + acc.row0(0) + 8 * p] = part[p];
      }
    };
    if (!rev) {
      dA.each([&](int r, int c, float& x) { A[r * (kC + 4) + c] = x * gates.between(r, c); });
      Acc<kC, NK> acc;
      acc.zero();
      acc.template mul<NV>(View{O, NV + 4, 1}, View{S, 1, NV + 4});
      acc.each([&](int r, int, float& x) { x *= gates.head[r]; });
      row_flow(acc, Q, &flow[0][0]);
      __syncthreads();
      acc.template mul<kC>(View{A, kC + 4, 1}, View{K, NK + 4, 1});
      acc.each([&](int r, int c, float& x) {
        if (r >= n) return;
        const size_t at = ((w.tok + t + r) * a.H + w.h) * NK + c;
        if (sp.dq_part) sp.dq_part[at] = a.scale * x;
        else dq[at] = a.scale * x;
      });
      if (threadIdx.x < n)
        sp.from[static_cast<size_t>(w.bh) * a.T + t + threadIdx.x] =
            a.scale * (flow[0][threadIdx.x] + flow[1][threadIdx.x]);
      __syncthreads();
      scale_rows<NV>(V, gates.tail);
      __syncthreads();
      update_state<NK, NV>(S, gates.sum, K, V);
      continue;
    }
    Acc<kC, kC> s;
    s.zero();
    s.template mul<NK>(View{Q, NK + 4, 1}, View{K, 1, NK + 4});
    s.each([&](int r, int c, float& x) {
      x *= a.scale * gates.between(r, c);
      A[r * (kC + 4) + c] = x;
    });
    __syncthreads();
    Acc<kC, NV> dvv;
    dvv.zero();
    dvv.template mul<NK>(View{K, NK + 4, 1}, View{S, NV + 4, 1});
    dvv.each([&](int r, int, float& x) { x *= gates.tail[r]; });
    dvv.template mul<kC>(View{A, 1, kC + 4}, View{O, NV + 4, 1});
    dvv.each([&](int r, int c, float& x) {
      if (r < n) dv[((w.tok + t + r) * a.H + w.h) * NV + c] = x;
    });
    __syncthreads();
    // M = s * dA into A, then its row and column sums
    dA.each([&](int r, int c, float& x) { A[r * (kC + 4) + c] *= x; });
    __syncthreads();
    if (threadIdx.x < 2 * kC) {
      const int r = threadIdx.x & (kC - 1);
      const int first = r & ~31, last = first + 32;
      float near = 0.f, far = 0.f;
      if (threadIdx.x < kC) {
        for (int c = 0; c < first; ++c) far += A[r * (kC + 4) + c];
        for (int c = first; c < r; ++c) near += A[r * (kC + 4) + c];
      } else {
        for (int c = r + 1; c < last; ++c) near += A[c * (kC + 4) + r];
        for (int c = last; c < kC; ++c) far += A[c * (kC + 4) + r];
      }
      flow[2 + (threadIdx.x >> 6)][r] = far;
      flow[4 + (threadIdx.x >> 6)][r] = near;
    }
    __syncthreads();
    dA.each([&](int r, int c, float& x) {
      A[r * (kC + 4) + c] = x * a.scale * gates.between(r, c);
    });
    Acc<kC, NK> dkk;
    dkk.zero();
    dkk.template mul<NV>(View{V, NV + 4, 1}, View{S, 1, NV + 4});
    dkk.each([&](int r, int, float& x) { x *= gates.tail[r]; });
    row_flow(dkk, K, &flow[0][0]);
    __syncthreads();
    dkk.template mul<kC>(View{A, 1, kC + 4}, View{Q, NK + 4, 1});
    dkk.each([&](int r, int c, float& x) {
      if (r >= n) return;
      const size_t at = ((w.tok + t + r) * a.H + w.h) * NK + c;
      if (sp.dk_part) sp.dk_part[at] = x;
      else dk[at] = x;
    });
    if (threadIdx.x < n) {
      const int r = threadIdx.x;
      const size_t p = static_cast<size_t>(w.bh) * a.T + t + r;
      const size_t plane = static_cast<size_t>(a.B) * a.H * a.T;
      sp.from[p + plane] = flow[2][r];
      sp.to[p] = flow[0][r] + flow[1][r];
      sp.to[p + plane] = flow[3][r];
      sp.near[p] = flow[4][r] - flow[5][r];
    }
    __syncthreads();
    if (threadIdx.x < kC) gates.head[threadIdx.x] *= a.scale;
    __syncthreads();
    scale_rows<NV>(O, gates.head);
    __syncthreads();
    update_state<NK, NV>(S, gates.sum, Q, O);
  }
  __syncthreads();
  if (!rev || blockIdx.x != 0) return;
  if (a.dh0) store_state<NK, NV>(S, a.dh0 + w.bh * st);
  if (a.h0) {   // <h0, D> where the gate's gradient starts
    float dot = 0.f;
    for (int i = threadIdx.x; i < NK * NV; i += kThreads)
      dot = fmaf(a.h0[w.bh * st + i], S[(i / NV) * (NV + 4) + i % NV], dot);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (lane == 0) flow[0][threadIdx.x >> 5] = dot;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < kThreads / 32; ++i) dot += flow[0][i];
      sp.first[w.bh] = dot;
    }
  }
}

template <class Kern>
cudaError_t run(Kern kern, const DecayArgs& a, const DecaySplit& sp, int segments, int z,
                size_t smem, cudaStream_t stream) {
  cudaError_t err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  kern<<<dim3(segments, a.B * a.H, z), kThreads, smem, stream>>>(a, sp);
  return cudaGetLastError();
}

constexpr size_t tile(int w) { return static_cast<size_t>(kC) * (w + 4) * 4; }
constexpr size_t state(int nk, int nv) { return static_cast<size_t>(nk) * (nv + 4) * 4; }

template <int NK, int NV>
struct F32 {
  static cudaError_t states(const DecayArgs& a, const DecaySplit& sp, bool rev, cudaStream_t s) {
    const size_t smem = state(NK, NV) + tile(NK) + tile(NV);
    return rev ? run(states_f32<NK, NV, true>, a, sp, sp.pieces - sp.slot_of(1), 1, smem, s)
               : run(states_f32<NK, NV, false>, a, sp, sp.states(a.dhT != nullptr), 1, smem, s);
  }
  static cudaError_t fwd(const DecayArgs& a, const DecaySplit& sp, cudaStream_t s) {
    return run(fwd_f32<NK, NV>, a, sp, sp.segments, 1,
               state(NK, NV) + 2 * tile(NK) + tile(NV) + tile(kC), s);
  }
  static cudaError_t bwd(const DecayArgs& a, const DecaySplit& sp, cudaStream_t s) {
    return run(bwd_f32<NK, NV>, a, sp, sp.segments, 2,
               state(NK, NV) + 2 * tile(NK) + 2 * tile(NV) + tile(kC), s);
  }
};

}  // namespace

#define GDR_WIDTHS(call)                                               \
  (a.nk == 64 ? (a.nv == 64 ? F32<64, 64>::call : F32<64, 128>::call)  \
              : (a.nv == 64 ? F32<128, 64>::call : F32<128, 128>::call))

cudaError_t launch_decay_states_f32(const DecayArgs& a, const DecaySplit& sp, bool reverse,
                                    cudaStream_t stream) {
  if ((reverse ? sp.pieces - sp.slot_of(1) : sp.states(a.dhT != nullptr)) < 1) return cudaSuccess;
  return GDR_WIDTHS(states(a, sp, reverse, stream));
}
cudaError_t launch_decay_fwd_f32(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  return GDR_WIDTHS(fwd(a, sp, stream));
}
cudaError_t launch_decay_bwd_f32(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  return GDR_WIDTHS(bwd(a, sp, stream));
}

}  // namespace gdr
