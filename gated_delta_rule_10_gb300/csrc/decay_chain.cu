// What joins the segments of the linear attention with a decay for each head:
// the chain of the segments' states, and the gate's gradient.
#include "common.cuh"
#include "decay.h"

namespace gdr {
namespace {

constexpr int kChainThreads = 256;

template <int kThreads>
__device__ __forceinline__ float block_sum(float x, float* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) s += red[i];
  return s;
}

// S_p = decay_{p-1} S_{p-1} + (piece p-1's own state), S_0 = h0; in place over
// the slots, each thread carrying one float4 of the state along the chain.
// Backward: D_p = decay_p D_{p+1} + (piece p's own gradient), D_P = dhT, and this
// block's part of <S_p, D_p> for every p >= 1.
// Bound by latency: a step is one load, one multiplication and one store, and slots
// are stored that later ones are loaded beside, so kBatch steps' loads are issued
// together before the first of their stores (1 x 29999 x 4 heads, 19 pieces: 6.4 us,
// step by step 11; backward 11 against 27, with one barrier for each batch's sums).
constexpr int kBatch = 8;

__device__ __forceinline__ float4 decayed4(float f, float4 s, float4 x) {
  return make_float4(decayed(f, s.x, x.x), decayed(f, s.y, x.y), decayed(f, s.z, x.z),
                     decayed(f, s.w, x.w));
}

template <bool BWD>
__global__ void __launch_bounds__(kChainThreads) chain_kernel(const DecayArgs a,
                                                              const DecaySplit sp) {
  constexpr int kWarps = kChainThreads / 32;
  __shared__ float red[2][kBatch][kWarps];
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const int bh = blockIdx.y, el = (blockIdx.x * kChainThreads + threadIdx.x) * 4;
  const size_t st = static_cast<size_t>(a.nk) * a.nv;
  float4* S = reinterpret_cast<float4*>(sp.S + bh * sp.slots * st + el);
  const float* decay = sp.decay + static_cast<size_t>(bh) * sp.pieces;
  const size_t step = st / 4;
  float4 s = a.h0 ? *reinterpret_cast<const float4*>(a.h0 + bh * st + el) : zero;
  S[0] = s;
  const int states = sp.states(a.dhT != nullptr);
  for (int p0 = 1; p0 <= states; p0 += kBatch) {
    float4 x[kBatch];
    float f[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (p0 + i <= states) {
        x[i] = S[(p0 + i) * step];
        f[i] = decay[p0 + i - 1];
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (p0 + i <= states) S[(p0 + i) * step] = s = decayed4(f[i], s, x[i]);
  }
  if (!BWD) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = sp.slot_of(1);
  float4* D = reinterpret_cast<float4*>(sp.D + bh * sp.slots * st + el);
  float4 d = a.dhT ? *reinterpret_cast<const float4*>(a.dhT + bh * st + el) : zero;
  for (int p0 = sp.pieces, half = 0; p0 >= first; p0 -= kBatch, half ^= 1) {
    float4 x[kBatch], y[kBatch];
    float f[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 - i;
      x[i] = y[i] = zero;
      f[i] = 0.f;
      if (p >= first) {
        if (p < sp.pieces) {
          x[i] = D[p * step];
          f[i] = decay[p];
        }
        // (the last state is not there where its gradient is zero)
        if (p <= states) y[i] = S[p * step];
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 - i;
      if (p < first) continue;
      if (p < sp.pieces) d = decayed4(f[i], d, x[i]);
      D[p * step] = d;
      float dot = y[i].x * d.x + y[i].y * d.y + y[i].z * d.z + y[i].w * d.w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
      if (lane == 0) red[half][i][warp] = dot;
    }
    __syncthreads();   // (the next batch writes the other half)
    if (threadIdx.x < kBatch && p0 - static_cast<int>(threadIdx.x) >= first) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += red[half][threadIdx.x][i];
      sp.dots[(static_cast<size_t>(bh) * sp.slots + p0 - threadIdx.x) * sp.parts + blockIdx.x] = sum;
    }
  }
}

__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  uint2 u = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
  *reinterpret_cast<uint2*>(p) = u;
}

// Gradients of a q and k head shared by several heads: the sum of theirs, by CTAs
// `cta` of `ctas`. It needs nothing of the gate's gradient and shares its launch
// (2 x 777 x 4 heads: 65 us, as a launch of its own 68).
template <typename T>
__device__ __forceinline__ void shared_grad(const DecayArgs& a, const DecaySplit& sp, size_t cta,
                                            size_t ctas) {
  const int r = a.H / a.Hk, shift = a.nk == 64 ? 4 : 5;   // float4s of a head, log2
  const size_t n4 = static_cast<size_t>(a.B) * a.T * a.Hk << shift;
  for (size_t i = cta * blockDim.x + threadIdx.x; i < 2 * n4; i += ctas * blockDim.x) {
    const bool key = i >= n4;
    const size_t j = key ? i - n4 : i, head = j >> shift;   // token * Hk + shared head
    const int c = static_cast<int>(j & ((1u << shift) - 1)) * 4;
    const float* src = (key ? sp.dk_part : sp.dq_part) + head * r * a.nk + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int n = 0; n < r; ++n) {
      const float4 x = *reinterpret_cast<const float4*>(src + static_cast<size_t>(n) * a.nk);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    store4(static_cast<T*>(key ? a.dk : a.dq) + head * a.nk + c, s);
  }
}

// The gate's gradient. With c the product <S, D> at a block's end (32 tokens),
//   dg_t = c + sum over the block's j >= t of (from_j - to_j + near_j),
//   <S, D> at its start = c - sum of to + sum of from.
// The near terms of a block sum to zero, so they stay out of what is passed on,
// and with them the rounding of the block's largest products. A block whose decay
// is below 2^-30 passes nothing on (what crosses it is 2^-30 of <S, D>): c is then
// its sum of to, and the start's its sum of from.
// So c is known at both ends of every run of blocks between such blocks and the
// segment's edges (from the states there, and from the sequence's own start). What
// the blocks' sums pass on, with rounding that gathers like a random walk, misses the
// far end by a little; the miss is spread over the run's blocks by the variance of what
// each may have rounded: the squares of its terms, of their sums and of c. (A large
// gradient of the last state is felt in the last blocks alone, but what those round is
// passed on to all: 4096 tokens of a fixed decay in fp32 missed its gradient by 5e-5 with
// the same share for every block.) A clearing token's gradient is 0.
constexpr int kMaxBlocks = 128;   // blocks per segment: 4096 tokens
constexpr int kMaxFlows = 3;      // two column slices and the pairs
constexpr int kGateThreads = 1024;

template <typename T>
__global__ void __launch_bounds__(kGateThreads) gate_grad_kernel(const DecayArgs a,
                                                                  const DecaySplit sp) {
  if (blockIdx.z > 0) {
    const size_t plane = static_cast<size_t>(gridDim.x) * gridDim.y;
    shared_grad<T>(a, sp, (blockIdx.z - 1) * plane + blockIdx.y * gridDim.x + blockIdx.x,
                   (gridDim.z - 1) * plane);
    return;
  }
  constexpr int kWarps = kGateThreads / 32;
  constexpr int kMine = kMaxBlocks / kWarps;   // blocks per warp
  constexpr float kMost = 1e36f;   // of a block's variance, that a run's is finite
  __shared__ float s_from[kMaxBlocks], s_to[kMaxBlocks], s_c[kMaxBlocks];
  __shared__ float s_var[kMaxBlocks], s_after[kMaxBlocks];   // a block's variance, and that
                                                             // of its run's later blocks
  __shared__ int s_keep[kMaxBlocks], s_run[kMaxBlocks];
  __shared__ float run_share[kMaxBlocks + 1];   // a run's miss over its variance
  __shared__ float red[kWarps];
  const int seg = blockIdx.x, bh = blockIdx.y, b = bh / a.H, h = bh % a.H;
  const int t0 = seg * sp.seg_len, t1 = min(a.T, t0 + sp.seg_len);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t plane = static_cast<size_t>(a.B) * a.H * a.T;
  const int blocks = (t1 - t0 + 31) / 32;
  bool clear[kMine];
  float suf[kMine];   // the block's sum from this token on
  float gs[kMine], fs[kMine], es[kMine], ls[kMine];
  // (all of a warp's loads before the first use: the backward of 4 x 4096 x 16 takes
  // 360 us, one block after another 367)
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int t = t0 + (warp + m * kWarps) * 32 + lane;
    gs[m] = fs[m] = es[m] = ls[m] = 0.f;
    if (t < t1) {
      gs[m] = a.per_head ? a.g[h] : a.g[(static_cast<size_t>(b) * a.T + t) * a.H + h];
      const size_t p = static_cast<size_t>(bh) * a.T + t;
#pragma unroll
      for (int i = 0; i < kMaxFlows; ++i)
        if (i < sp.flows) {
          fs[m] += sp.from[p + i * plane];
          es[m] += sp.to[p + i * plane];
        }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (i < sp.nears) ls[m] += sp.near[p + i * plane];
    }
  }
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int blk = warp + m * kWarps;
    float g = gs[m], f = fs[m], e = es[m], var = f * f + e * e;
    const float l = ls[m];
    clear[m] = g <= kDecayReset;
    suf[m] = f - e + l;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      f += __shfl_xor_sync(0xffffffffu, f, off);
      e += __shfl_xor_sync(0xffffffffu, e, off);
      g += __shfl_xor_sync(0xffffffffu, g, off);
      var += __shfl_xor_sync(0xffffffffu, var, off);
    }
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const float y = __shfl_down_sync(0xffffffffu, suf[m], off);
      if (lane + off < 32) suf[m] += y;
    }
    if (lane == 0 && blk < blocks) {
      s_from[blk] = f;
      s_to[blk] = e;
      s_var[blk] = fminf(var + (f * f + e * e), kMost);
      s_keep[blk] = !(g < -20.8f);   // (NaN keeps)
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    auto edge = [&](int slot) {   // <S, D> at a segment's edge
      float c = 0.f;
      if (sp.dots)
        for (int i = 0; i < sp.parts; ++i)
          c += sp.dots[(static_cast<size_t>(bh) * sp.slots + slot) * sp.parts + i];
      return c;
    };
    float c = edge(sp.slot_of(seg + 1));
    float start = 0.f;
    if (seg > 0) start = edge(sp.slot_of(seg));
    else if (a.h0)
      for (int i = 0; i < sp.firsts; ++i) start += sp.first[bh * sp.firsts + i];
    float after = 0.f;   // the variance of the run's blocks so far
    int run = 0;
    for (int blk = blocks - 1; blk >= 0; --blk) {
      const bool keep = s_keep[blk];
      const float f = s_from[blk], e = s_to[blk];
      const float var = fminf(s_var[blk] + c * c, kMost);
      s_c[blk] = keep ? c : e;
      s_run[blk] = keep ? run : kMaxBlocks;
      s_after[blk] = after;
      if (keep) {
        c += f - e;
        after += var;
      }
      // a run's far end is a block that passes nothing, or the segment's start
      if (!keep || blk == 0) {
        run_share[run++] = after > 1e-30f ? (c - (keep ? start : e)) / after : 0.f;
        after = 0.f;
      }
      if (!keep) c = f;
    }
    run_share[kMaxBlocks] = 0.f;
  }
  __syncthreads();
  float total = 0.f;
#pragma unroll
  for (int m = 0; m < kMine; ++m) {
    const int blk = warp + m * kWarps, t = t0 + blk * 32 + lane;
    if (t >= t1) continue;
    const float c = s_c[blk] - run_share[s_run[blk]] * s_after[blk];
    const float out = clear[m] ? 0.f : c + suf[m];
    if (a.per_head) total += out;
    else a.dg[(static_cast<size_t>(b) * a.T + t) * a.H + h] = out;
  }
  if (a.per_head) {
    const float s = block_sum<kGateThreads>(total, red);
    if (threadIdx.x == 0) sp.dg_part[static_cast<size_t>(bh) * sp.segments + seg] = s;
  }
}

// Sum over batches and segments of a fixed decay's gradient, one warp per head.
__global__ void __launch_bounds__(32) head_grad_kernel(const DecayArgs a, const DecaySplit sp) {
  const int h = blockIdx.x, n = a.B * sp.segments;
  float s = 0.f;
  for (int i = threadIdx.x; i < n; i += 32)
    s += sp.dg_part[(static_cast<size_t>(i / sp.segments) * a.H + h) * sp.segments +
                    i % sp.segments];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  if (threadIdx.x == 0) a.dg[h] = s;
}

}  // namespace

cudaError_t launch_decay_chain(const DecayArgs& a, const DecaySplit& sp, bool backward,
                               cudaStream_t stream) {
  const dim3 grid(a.nk * a.nv / (4 * kChainThreads), a.B * a.H);
  if (backward) chain_kernel<true><<<grid, kChainThreads, 0, stream>>>(a, sp);
  else chain_kernel<false><<<grid, kChainThreads, 0, stream>>>(a, sp);
  return cudaGetLastError();
}

cudaError_t launch_decay_gate_grad(const DecayArgs& a, const DecaySplit& sp, bool f32,
                                   cudaStream_t stream) {
  dim3 grid(sp.segments, a.B * a.H, 1);
  if (sp.dq_part) {   // two float4s a thread, up to 16 planes
    const size_t work = static_cast<size_t>(a.B) * a.T * a.Hk * (a.nk / 4);
    const size_t planes = work / (static_cast<size_t>(kGateThreads) * grid.x * grid.y) + 1;
    grid.z += static_cast<unsigned>(planes < 16 ? planes : 16);
  }
  if (f32) gate_grad_kernel<float><<<grid, kGateThreads, 0, stream>>>(a, sp);
  else gate_grad_kernel<__nv_bfloat16><<<grid, kGateThreads, 0, stream>>>(a, sp);
  if (a.per_head) head_grad_kernel<<<a.H, 32, 0, stream>>>(a, sp);
  return cudaGetLastError();
}

}  // namespace gdr
