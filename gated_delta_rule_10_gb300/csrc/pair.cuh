// Pairs of fp32 in one 64-bit register pair, which one instruction handles, and the
// exponential, reciprocal and sigmoid that the block operators use.
#pragma once

#include <cuda_runtime.h>

namespace gdr {

constexpr float kLog2e = 1.4426950408889634f;

using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f32x2 both(float v) { return pair(v, v); }
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
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 1 / (1 + e^-x): far below zero e^-x overflows and the result is zero, as it is in fp32
// from x = -104 on (-88 with the reciprocal's flushing).
__device__ __forceinline__ float sigmoid(float x) {
  return rcp_fast(1.f + exp2_fast(-kLog2e * x));
}
__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  float lo, hi;
  split(add2(both(1.f), exp2_pair(mul2(x, both(-kLog2e)))), lo, hi);
  return pair(rcp_fast(lo), rcp_fast(hi));
}
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

}  // namespace gdr
