// Shared parts of the tensor-core kernels of the linear attention with a decay
// for each head (bf16, chunks of 128 tokens): the chunk's decay factors, bounded
// waits and the conversion of a row-scaled operand into two bf16 tiles.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "decay.h"
#include "tc.cuh"

namespace gdr {
namespace dtc {

constexpr int kC = 128;             // tokens per chunk
constexpr uint32_t kTile = 16384;   // 128 rows of 64 bf16 columns, 128-byte swizzle

// Decay factors of one chunk. Four blocks of 32 tokens; a pair (r, i) in
// different blocks has e^{G_r - G_i} = row[r] * col[b][i] with b the block of r,
// both factors sums over disjoint spans (no difference of long sums), and a pair
// within a block takes the exponential of the difference of block-local sums.
// A clearing token (kDecayReset) leaves the sums and zeroes the factors that
// span it.
__device__ __forceinline__ int col_at(int b) { return 16 * b * (b - 1); }   // 0, 32, 96
struct Gates {
  float loc[kC];        // log2 of the decay from the block's start through r
  uint32_t allow[kC];   // bit i: token i of r's block reaches r (backward: r reaches i)
  float row[kC];        // decay from the block's start through r
  float col[192];       // col[col_at(b) + i]: decay from after i through the end of block b-1
  float head[kC];       // decay from the chunk's start through r
  float tail[kC];       // decay from after i through the chunk's end
  float sum;            // log of the whole chunk's decay
  float all;            // that decay (decay_code)
  float pad[2];
};
// For sums over the pairs in fp32 (the gate's gradient), with what the rounding of loc
// leaves: tokens near -100 that do not clear take the sums to thousands, where a
// difference of two fp32 values is off by 2e-4. (A . D is rounded to bf16, 2e-3, and does
// without: with it the forward of 4 x 4096 x 16 x 128 took 80 us instead of 68.)
struct PairGates : Gates {
  float low[kC];
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 values in one 64-bit register pair: one instruction for both.
using F2 = unsigned long long;
__device__ __forceinline__ F2 pack2(float a, float b) {
  F2 d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ void unpack2(F2 d, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(d));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint32_t round2(F2 x) {
  float a, b;
  unpack2(x, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ F2 widen2(uint32_t w) {
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// 16 columns at each of two places, one wait for both.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, float (&u)[16],
                                            float (&v)[16]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%32];\n"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%33];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(ta), "r"(tb)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    u[i] = __uint_as_float(r[i]);
    v[i] = __uint_as_float(r[16 + i]);
  }
}

// The log-decays of this lane's tokens 32 j + lane (0 past n).
__device__ __forceinline__ void read_gates(float (&x)[4], const DecayArgs& a, size_t tok, int h,
                                           int n) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int r = 32 * j + lane;
    x[j] = r < n ? (a.per_head ? a.g[h] : __ldg(a.g + (tok + r) * a.H + h)) : 0.f;
  }
}

// hi + lo += x + y, the sum's rounding error kept.
__device__ __forceinline__ void add_pair(float& hi, float& lo, float x, float y) {
  const float s = hi + x, part = s - hi;
  lo += ((hi - (s - part)) + (x - part)) + y;
  hi = s;
}

__device__ __forceinline__ float exp_fast(float x) { return exp2_fast(x * 1.4426950408889634f); }

// One warp turns the chunk's log-decays into its factors, a block of 32 tokens
// per lane and register, so that the four blocks' shuffles overlap. Running sums
// are taken from both ends: a factor never comes from a difference of sums, and
// the error of exp_fast, |x| 2^-23, is small where the factor is not.
template <bool REV, class G>
__device__ __forceinline__ void fill_gates(G& s, const float (&x)[4]) {
  constexpr bool kLow = std::is_same<G, PairGates>::value;
  const int lane = threadIdx.x & 31;
  const uint32_t to = 0xffffffffu >> (31 - lane);   // tokens up to this one
  float up[4], low[4] = {}, down[4], total[4];
  uint32_t clears[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const bool clear = x[b] <= kDecayReset;
    clears[b] = __ballot_sync(0xffffffffu, clear);
    up[b] = down[b] = clear ? 0.f : x[b];
  }
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float u = __shfl_up_sync(0xffffffffu, up[b], off);
      const float d = __shfl_down_sync(0xffffffffu, down[b], off);
      if constexpr (kLow) {
        const float l = __shfl_up_sync(0xffffffffu, low[b], off);
        add_pair(up[b], low[b], lane >= off ? u : 0.f, lane >= off ? l : 0.f);
      } else {
        up[b] += lane >= off ? u : 0.f;
      }
      down[b] += lane + off < 32 ? d : 0.f;
    }
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    total[b] = __shfl_sync(0xffffffffu, up[b], 31);
    if (clears[b]) total[b] = -INFINITY;
    down[b] = __shfl_down_sync(0xffffffffu, down[b], 1);
    if (lane == 31) down[b] = 0.f;
    const uint32_t before = clears[b] & to;
    const float log2e = 1.4426950408889634f, loc = up[b] * log2e;
    s.loc[32 * b + lane] = loc;
    if constexpr (kLow) s.low[32 * b + lane] = fmaf(up[b], log2e, -loc) + low[b] * log2e;
    const uint32_t behind = clears[b] & ~to;
    s.allow[32 * b + lane] =
        REV ? (0xffffffffu << lane) & (behind ? (1u << (__ffs(behind) - 1)) - 1u : 0xffffffffu)
            : to & (0xffffffffu << (before ? 31 - __clz(before) : 0));
    if (before) up[b] = -INFINITY;
    if (behind) down[b] = -INFINITY;
  }
  float pre = 0.f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    const int r = 32 * b + lane;
    s.row[r] = exp_fast(up[b]);
    s.head[r] = exp_fast(pre + up[b]);
    float e = down[b];
#pragma unroll
    for (int w = b + 1; w < 4; ++w) {
      s.col[col_at(w) + r] = exp_fast(e);
      e += total[w];
    }
    s.tail[r] = exp_fast(e);
    pre += total[b];
  }
  if (lane == 0) {
    s.sum = pre;
    s.all = decay_code(pre);
  }
}

// Bounded mbarrier wait that also gives up once another role has aborted.
__device__ __noinline__ bool wait_long(uint32_t mbar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (uint32_t i = 0; i < tc::kMaxPolls; ++i) {
    if (tc::mbar_try_wait(mbar, parity, tc::kSuspendNs)) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = 1;
  return false;
}
// The first poll is in line and lets the hardware choose how long it may sleep.
__device__ __forceinline__ bool wait(uint32_t mbar, uint32_t parity, volatile int* abort_flag) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(mbar), "r"(parity)
      : "memory");
  return done || wait_long(mbar, parity, abort_flag);
}
// The same for a whole warp, with one answer. Every lane polls: with one lane
// polling in a branch of its own, a hand-over took several times as long.
__device__ __forceinline__ bool warp_wait(uint32_t mbar, uint32_t parity, volatile int* abort_flag) {
  return __all_sync(0xffffffffu, wait(mbar, parity, abort_flag));
}
// One arrival for a whole warp.
__device__ __forceinline__ void warp_arrive(uint32_t mbar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::mbar_arrive(mbar);
}

// Products issued by the lane with `go` set of a converged warp. The whole warp
// runs the issuing code, so that descriptors stay in uniform registers; from a
// branch of one lane every operand of every product is moved there first
// (measured: 130 cycles a product).
__device__ __forceinline__ void mma_if(uint32_t go, uint32_t d, uint64_t x, uint64_t y,
                                       uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(x), "l"(y), "r"(id), "r"(accumulate), "r"(go));
}
__device__ __forceinline__ void mma_ta_if(uint32_t go, uint32_t d, uint32_t x, uint64_t y,
                                          uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(x), "l"(y), "r"(id), "r"(accumulate), "r"(go));
}
__device__ __forceinline__ void commit_if(uint32_t go, uint32_t mbar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(
          mbar),
      "r"(go)
      : "memory");
}

__device__ __forceinline__ uint4 lds4(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(addr)
               : "memory");
  return u;
}
__device__ __forceinline__ void sts4(uint32_t addr, const uint32_t (&u)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(u[0]), "r"(u[1]),
               "r"(u[2]), "r"(u[3])
               : "memory");
}

// x in three bf16 terms (24 bits): hi, and what it leaves, and what that leaves.
struct Terms {
  uint32_t hi, mid, lo;
};
__device__ __forceinline__ Terms terms_of(F2 x) {
  const F2 minus = pack2(-1.f, -1.f);
  Terms t;
  t.hi = round2(x);
  x = fma2(widen2(t.hi), minus, x);
  t.mid = round2(x);
  t.lo = round2(fma2(widen2(t.mid), minus, x));
  return t;
}

// Two pieces of 16 bytes (16 columns from column 8 c) times f, into row `r` of TERMS
// tiles `apart` bytes from one another: two leave 2.4e-6 of the state they feed,
// three 1e-7.
template <int TERMS>
__device__ __forceinline__ void split_pair(const uint4 (&u)[2], uint32_t dst, uint32_t apart, int r,
                                           int c, float f) {
  const F2 ff = pack2(f, f);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t w[4] = {u[p].x, u[p].y, u[p].z, u[p].w};
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Terms t = terms_of(mul2(widen2(w[i]), ff));
      hi[i] = t.hi;
      mid[i] = t.mid;
      lo[i] = t.lo;
    }
    const uint32_t d = dst + r * 128 + (((c + p) ^ (r & 7)) << 4);
    sts4(d, hi);
    sts4(d + apart, mid);
    if (TERMS == 3) sts4(d + 2 * apart, lo);
  }
}
// The same from row `r` of a tile with 64 bf16 columns.
template <int TERMS>
__device__ __forceinline__ void split_row(uint32_t src, uint32_t dst, uint32_t apart, int r, int c,
                                          float f) {
  uint4 u[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) u[p] = lds4(src + r * 128 + (((c + p) ^ (r & 7)) << 4));
  split_pair<TERMS>(u, dst, apart, r, c, f);
}

// 64 fp32 values as one row of a swizzled bf16 tile with 128-byte rows; with ALL as
// three tiles `apart` bytes from one another.
template <bool ALL>
__device__ __forceinline__ void round_row(uint32_t dst, uint32_t apart, int r,
                                          const float (&x)[64]) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint32_t d = dst + r * 128 + ((c ^ (r & 7)) << 4);
    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const F2 v = pack2(x[8 * c + 2 * i], x[8 * c + 2 * i + 1]);
      if (ALL) {
        const Terms t = terms_of(v);
        hi[i] = t.hi;
        mid[i] = t.mid;
        lo[i] = t.lo;
      } else {
        hi[i] = round2(v);
      }
    }
    sts4(d, hi);
    if (ALL) {
      sts4(d + apart, mid);
      sts4(d + 2 * apart, lo);
    }
  }
}

// S = decay * S + (hi + rest), as decayed() does, two at a time, from 128 accumulator
// columns [hi 64 | the other terms 64].
__device__ __forceinline__ void add_state(float (&S)[64], float all, uint32_t taddr) {
  const float near = signbit(all) ? 1.f : 0.f;
  const F2 g = pack2(all, all), c = pack2(near, near);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    float hi[16], lo[16];
    tmem_ld16x2(taddr + 16 * p, taddr + 64 + 16 * p, hi, lo);
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      float &a = S[16 * p + j], &b = S[16 * p + j + 1];
      const F2 s = pack2(a, b), p2 = add2(pack2(hi[j], hi[j + 1]), pack2(lo[j], lo[j + 1]));
      unpack2(fma2(g, s, fma2(c, s, p2)), a, b);
    }
  }
}

// 64 state values of one row, `step` elements apart; null: zeros.
__device__ __forceinline__ void read_row(float (&S)[64], const float* src, int step) {
#pragma unroll
  for (int j = 0; j < 64; ++j) S[j] = src ? src[static_cast<size_t>(j) * step] : 0.f;
}
__device__ __forceinline__ void write_row(const float (&S)[64], float f, float* dst) {
#pragma unroll
  for (int j = 0; j < 64; j += 4)
    *reinterpret_cast<float4*>(dst + j) =
        make_float4(f * S[j], f * S[j + 1], f * S[j + 2], f * S[j + 3]);
}

}  // namespace dtc
}  // namespace gdr
