// Device helpers of the state space recurrence's kernels: the step size and the channels of
// a CTA.
#pragma once

#include "pair.cuh"
#include "state_space.h"
#include "vec_io.cuh"

namespace gdr {

// log(1 + e^v) = max(v, 0) + log(1 + q), q = e^-|v| in (0, 1], and with s = q / (2 + q)
// log(1 + q) = 2 atanh(s) = 2 (s + s^3 / 3 + s^5 / 5 + ...), s <= 1/3: six terms leave
// 1.4e-7 of it, and small steps keep all their digits (1 + q would not). q is 2^(-|v| log2 e)
// times 1 + what the product's rounding leaves of |v| (at v = -7 three bits).
__device__ __forceinline__ f32x2 softplus2(f32x2 v) {
  constexpr float kLn2 = 0.6931471805599453f;
  float v0, v1, r0, r1;
  split(v, v0, v1);
  // (q is zero from -88 on, and the bound keeps infinities out of the products)
  const f32x2 n = pair(fmaxf(-fabsf(v0), -120.f), fmaxf(-fabsf(v1), -120.f));
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r0) : "f"(v0));
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r1) : "f"(v1));
  const f32x2 e = mul2(n, both(kLog2e));
  f32x2 q = exp2_pair(e);
  q = fma2(q, fma2(e, both(-kLn2), n), q);
  float d0, d1;
  split(add2(q, both(2.f)), d0, d1);
  const f32x2 s = mul2(q, pair(rcp_fast(d0), rcp_fast(d1))), s2 = mul2(s, s);
  f32x2 p = fma2(s2, both(2.f / 11.f), both(2.f / 9.f));
  p = fma2(p, s2, both(2.f / 7.f));
  p = fma2(p, s2, both(2.f / 5.f));
  p = fma2(p, s2, both(2.f / 3.f));
  p = fma2(p, s2, both(2.f));
  return fma2(p, s, pair(r0, r1));
}
__device__ __forceinline__ float softplus(float v) {
  float lo, hi;
  split(softplus2(both(v)), lo, hi);
  return lo;
}

// The decay of one token, 2^(a u) with a = log2(e) A. The exponential unit's results are low by
// 0.1 of 2^-24 on average for exponents from 0 to -2^-8 and by 0.3 to 0.45 from there to -1, which
// a state gathers from every token that it keeps; the exponent's rounding is to both sides. 1e-8
// more in the exponent, which the product's instruction adds, leaves 0.03 of the former and 0.1 to
// 0.35 of the latter, and 2^0 is 1 all the same: the end states of 8 x 4096 tokens x 8192 channels
// with steps of 1e-5 to 1e-3 come to 4.2e-6 of 64 bits instead of 2.8e-5. Growing states, where
// the unit errs to the other side (0.15 of 2^-24 on average up to 2^-8), get 0.12 more: a choice
// by the sign of A takes registers that the gradients' kernel would spill.
__device__ __forceinline__ f32x2 decay2(f32x2 a, f32x2 u) {
  return exp2_pair(fma2(a, u, both(1e-8f)));
}

// 16 bytes from global to shared memory, and the wait for all of a thread's copies.
__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void copies_done() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}
// 8 elements of T, in 16-byte pieces.
template <typename T>
__device__ __forceinline__ void copy8(T* to, const T* from) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    copy16(reinterpret_cast<uint4*>(to) + i, reinterpret_cast<const uint4*>(from) + i);
}
template <typename T>
__device__ __forceinline__ void read8(const T* p, f32x2 (&x)[4]) {   // from shared memory
  if constexpr (sizeof(T) == 4) {
    const ulonglong2 a = reinterpret_cast<const ulonglong2*>(p)[0];
    const ulonglong2 b = reinterpret_cast<const ulonglong2*>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
}
__device__ __forceinline__ void write8(float* p, const f32x2 (&x)[4]) {   // to shared memory
  reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(x[0], x[1]);
  reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(x[2], x[3]);
}

template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const f32x2 (&x)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(x[i], f[2 * i], f[2 * i + 1]);
  store8(p, f);
}

// Lets a kernel have `BYTES` of shared memory.
template <auto Kern, int BYTES>
cudaError_t allow_shared() {
  static_assert(BYTES <= 232448, "shared memory of one CTA");
  return cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
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

}  // namespace gdr
