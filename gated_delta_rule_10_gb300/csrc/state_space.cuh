// Device helpers of the state space recurrence's kernels: pairs of fp32 in one register
// pair, exponentials, the step size and its slope, and the channels of a CTA.
#pragma once

#include "state_space.h"
#include "vec_io.cuh"

namespace gdr {

constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 numbers handled by one instruction.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(f32x2 v) {
  float lo, hi;
  split(v, lo, hi);
  return lo + hi;
}

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f32x2 exp2_pair(f32x2 v) {
  float lo, hi;
  split(v, lo, hi);
  return pair(exp2_fast(lo), exp2_fast(hi));
}

__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.f, 1.f + exp2_fast(-kLog2e * x));
}
// x sigmoid(x) and its slope
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ float silu_slope(float x) {
  const float s = sigmoid(x);
  return s * fmaf(x, 1.f - s, 1.f);
}

// e^v for v <= 0 to about 2^-22 of it: the product with log2(e) keeps what its rounding
// leaves (v = -7 would lose three bits by it).
__device__ __forceinline__ float exp_kept(float v) {
  const float hi = v * kLog2e;
  // log2(e) - kLog2e = 1.925963e-8
  const float lo = fmaf(v, 1.9259630e-8f, fmaf(v, kLog2e, -hi));
  const float e = exp2_fast(hi);
  return v > -104.f ? fmaf(e, lo * 0.6931471805599453f, e) : 0.f;
}

// log(1 + e^v) = max(v, 0) + log(1 + q), q = e^-|v| in (0, 1], and with s = q / (2 + q)
// log(1 + q) = 2 atanh(s) = 2 (s + s^3 / 3 + s^5 / 5 + ...), s <= 1/3: nine terms leave
// 1e-9 of it, and small steps keep all their digits (1 + q would not).
__device__ __forceinline__ float softplus(float v) {
  const float q = exp_kept(-fabsf(v));
  const float s = __fdividef(q, 2.f + q), s2 = s * s;
  float p = 2.f / 17.f;
  p = fmaf(p, s2, 2.f / 15.f);
  p = fmaf(p, s2, 2.f / 13.f);
  p = fmaf(p, s2, 2.f / 11.f);
  p = fmaf(p, s2, 2.f / 9.f);
  p = fmaf(p, s2, 2.f / 7.f);
  p = fmaf(p, s2, 2.f / 5.f);
  p = fmaf(p, s2, 2.f / 3.f);
  p = fmaf(p, s2, 2.f);
  return v != v ? v : fmaf(p, s, v > 0.f ? v : 0.f);
}

// The channels of a CTA: `width` at most, all of one group.
struct Channels {
  int first, end, group;
  __device__ __forceinline__ Channels(const SpaceArgs& a, int width, int block) {
    const int each = a.D / a.G, per = (each + width - 1) / width;
    group = block / per;
    first = group * each + (block % per) * width;
    end = min(first + width, (group + 1) * each);
  }
};

// The state entering segment s, states [d * N + n, + 4) of batch row b, from the slots of
// `sp.h` (see there): what the segments before it leave, chained.
__device__ __forceinline__ void chain_states(const SpaceArgs& a, const SpaceSplit& sp, int b, int s,
                                             int d, int n, const float (&A2)[4], float (&h)[4]) {
  const size_t state = static_cast<size_t>(a.D) * a.N;
  const float* slot = sp.h + static_cast<size_t>(b) * sp.segments * state +
                      static_cast<size_t>(d) * a.N + n;
  const int from = s == 0 ? 0 : 1;
  const float4 v = *reinterpret_cast<const float4*>(slot + from * state);
  h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
  for (int i = 2; i <= s; ++i) {
    const float u = sp.total[(static_cast<size_t>(b) * sp.segments + i - 1) * a.D + d];
    const bool cleared = sp.cleared[b * sp.segments + i - 1] != 0;
    const float4 w = *reinterpret_cast<const float4*>(slot + i * state);
    const float add[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      h[j] = cleared ? add[j] : fmaf(exp2_fast(A2[j] * u), h[j], add[j]);
  }
}

}  // namespace gdr
