// Linear attention with a decay for each head, chunked, for bf16 inputs: the
// forward and the segments' own states on tcgen05.
//
// With chunks of 128 tokens, D_ri = e^{G_r - G_i} for i <= r and 64 value columns
// per CTA, a chunk takes four products:
//   A  = Q K^T                        (128 x 128, K = d_k)
//   O1 = Q S_n                        (128 x 64,  K = d_k)
//   O2 = (A . D) V                    (128 x 64,  K = 128, A . D from tensor memory)
//   P  = K^T [V'hi | V'lo]            (d_k x 128, K = 128), V' = e^{G_C - G_i} V
//   o  = s (e^{G_r} O1 + O2),   S_{n+1} = e^{G_C} S_n + P_hi + P_lo.
// q, k and v go from TMA to the tensor cores as they are. A . D and the S of the
// read-out are rounded to bf16 (o is rounded to bf16 anyway); the decayed V' is
// split into two bf16 terms because it enters the fp32 state, whose error would
// otherwise be bf16's. The two terms sit side by side, one N = 128 product.
//
// Only S_{n+1} <- S_n is a chain, and it holds no product: P of any chunk can be
// ready before S is. So the tensor pipe can run without a gap; the products of a
// chunk are issued as P(n), A(n+1), O2(n), O1(n+1), which gives each role (the
// mask on A, the state, the read-out) about one chunk's time, and the loads one
// chunk's lead: q is free after O1, k after P, v after O2.
// The two column halves of a head re-read q and k (from L2) and repeat A.
#include "decay_tc.cuh"
#include "tma.h"

namespace gdr {
namespace {

using namespace dtc;

// ------------------------------------------------------------------ forward

constexpr int kFwdThreads = 512;   // 3 x 128: mask, state, read-out; loads; products; gates (2)
constexpr uint32_t kCols = 512;
// tensor-memory columns: two buffers of [A 128] (A . D as bf16 overwrites columns
// 0..63, O2 columns 64..127), two of O1, and P
constexpr uint32_t cA = 0, cO1 = 256, cP = 384;

enum : uint32_t {   // mbarriers, each a pair for even and odd chunks
  bQK = 0, bV = 4,                   // tiles landed
  bMA = 6, bMO1 = 8, bMO2 = 10, bMP = 12,   // products complete
  bMask = 14, bSplit = 16, bState = 18, bFree = 20,
  bGates = 22, bGFree = 26,          // four each: a ring of four chunks' gates
  bEnd = 30, kBars = 32
};

template <int NK>
struct FwdSmem {
  static constexpr uint32_t kWide = NK / 64 * kTile;
  static constexpr uint32_t oQ = 0, oK = oQ + 2 * kWide, oV = oK + 2 * kWide, oSplit = oV + 2 * kTile,
                            oS = oSplit + 2 * kTile, oGates = oS + NK * 128,
                            oBar = oGates + 4 * sizeof(Gates), oSlot = oBar + 8 * kBars,
                            oAbort = oSlot + 4, bytes = oAbort + 12;
  static constexpr uint32_t launch = bytes + 1024;   // room to align the base
};

template <int NK>
__global__ void __launch_bounds__(kFwdThreads, 1)
    decay_fwd_tc(const DecayArgs a, const DecaySplit sp, const __grid_constant__ CUtensorMap tq,
                 const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv) {
  using L = FwdSmem<NK>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = a.nv / 64, slice = blockIdx.x % slices, seg = blockIdx.x / slices;
  const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int t0 = seg * sp.seg_len, t1 = min(a.T, t0 + sp.seg_len);
  const int cnt = (t1 - t0 + kC - 1) / kC;
  const size_t tok0 = static_cast<size_t>(b) * a.T + t0;
  auto bar = [&](uint32_t i, int n) { return sb + L::oBar + 8 * (i + (n & 1)); };
  auto par = [](int n) { return static_cast<uint32_t>(n >> 1) & 1u; };
  auto bar4 = [&](uint32_t i, int n) { return sb + L::oBar + 8 * (i + (n & 3)); };
  auto par4 = [](int n) { return static_cast<uint32_t>(n >> 2) & 1u; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oAbort);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::oSlot);
  auto gates = [&](int n) -> Gates& {
    return *reinterpret_cast<Gates*>(smem + L::oGates + (n & 3) * sizeof(Gates));
  };

  if (warp == 13) tc::tmem_alloc(smem_u32(slot), kCols);
  if (tid == 0) {
    for (uint32_t i = 0; i < kBars; ++i) {
      uint32_t count = i < bV ? 2 : 1;   // q and k land on one barrier
      if (i >= bMask && i < bGates) count = i == bSplit || i == bSplit + 1 ? 8 : 4;   // warps
      if (i >= bGFree && i < bEnd) count = 8;
      tc::mbar_init(sb + L::oBar + 8 * i, count);
    }
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  const int quad = warp & 3, row = 32 * quad + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16);

  // tiles of chunk n into their slots; the roles that see a slot's last reader
  // finish ask for the next tile themselves (one lane)
  auto load_wide = [&](uint32_t base, const CUtensorMap* m, int n) {
    tc::mbar_arrive_expect_tx(bar(bQK, n), L::kWide);
#pragma unroll
    for (int blk = 0; blk < NK / 64; ++blk)
      tc::tma_load_4d(sb + base + (n & 1) * L::kWide + blk * kTile, m, 64 * blk, hk, t0 + n * kC, b,
                      bar(bQK, n));
  };
  auto load_v = [&](int n) {
    tc::mbar_arrive_expect_tx(bar(bV, n), kTile);
    tc::tma_load_4d(sb + L::oV + (n & 1) * kTile, &tv, 64 * slice, h, t0 + n * kC, b, bar(bV, n));
  };
  // half of the columns of this lane's token of V'; its last reader is P(n - 1),
  // whose completion the caller has waited for
  auto split = [&](int n, int half) {
    if (!warp_wait(bar4(bGates, n), par4(n), abort_flag) || !warp_wait(bar(bV, n), par(n), abort_flag))
      return false;
    split_row(smem + L::oV + (n & 1) * kTile, smem + L::oSplit, row, 4 * half, gates(n).tail[row]);
    tc::fence_proxy_async();
    warp_arrive(bar(bSplit, n));
    return true;
  };

  if (warp < 4) {
    // ---------------------------------------------- A . D, one token per lane
    for (int n = 0; n < cnt; ++n) {
      const bool ok = warp_wait(bar4(bGates, n), par4(n), abort_flag) &&
                      warp_wait(bar(bMA, n), par(n), abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const Gates& g = gates(n);
      const uint32_t ta = tl + cA + (n & 1) * 128;
      const float lr = g.loc[row], fr = g.row[row];
      const uint32_t allow = g.allow[row];
#pragma unroll 1
      for (int cb = 0; cb < 4; ++cb) {
        uint32_t r[16];
        if (cb > quad) {
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = 0u;
        } else {
          float x[32];
          tc::tmem_ld32(ta + 32 * cb, x);
          const float* f = g.col + col_at(quad) + 32 * cb;
          if (cb == quad) {
            f = g.loc + 32 * cb;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 v = *reinterpret_cast<const float4*>(f + i);
              const float c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float e = exp2_fast(lr - c[j]);
                x[i + j] = (allow >> (i + j)) & 1u ? x[i + j] * e : 0.f;
              }
              r[i / 2] = pack_bf16x2(x[i], x[i + 1]);
              r[i / 2 + 1] = pack_bf16x2(x[i + 2], x[i + 3]);
            }
          } else {
            const F2 ff = pack2(fr, fr);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(f + i);
              r[i / 2] = round2(mul2(pack2(x[i], x[i + 1]), mul2(ff, c.x)));
              r[i / 2 + 1] = round2(mul2(pack2(x[i + 2], x[i + 3]), mul2(ff, c.y)));
            }
          }
        }
        tc::tmem_st16(ta + 16 * cb, r);   // over columns already read
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(bar(bMask, n));
    }
  } else if (warp < 8) {
    // ---------------------------------------------- the state, one key channel per
    // lane, and half of V' 
    int nq = 0, nk = 0;   // (tid 128) tiles requested
    if (tid == 128)
      for (; nq < min(2, cnt); ++nq, ++nk) {
        load_wide(L::oQ, &tq, nq);
        load_wide(L::oK, &tk, nk);
      }
    __syncwarp();
    const bool mine = row < NK;
    const size_t st = static_cast<size_t>(NK) * a.nv;
    const float* start = sp.segments > 1 ? sp.S + (static_cast<size_t>(bh) * sp.slots + seg) * st
                                         : (a.h0 ? a.h0 + bh * st : nullptr);
    float S[64];
    read_row(S, start && mine ? start + static_cast<size_t>(row) * a.nv + 64 * slice : nullptr);
    if (mine) round_row(smem + L::oS, row, S);
    tc::fence_proxy_async();
    warp_arrive(bar(bState, 0));
    bool ok = split(0, 0);
    for (int n = 0; ok && n < cnt; ++n) {
      ok = warp_wait(bar(bMP, n), par(n), abort_flag);
      if (!ok) break;
      if (tid == 128 && n + 2 < cnt && wait(bar(bMA, n), par(n), abort_flag)) {
        load_wide(L::oK, &tk, n + 2);   // k's readers A(n) and P(n) are done
        nk = n + 3;
      }
      __syncwarp();
      tc::fence_after_sync();
      const float all = gates(n).all;
      warp_arrive(bar4(bGFree, n));
      if (mine || NK == 128) add_state(S, all, tl + cP);
      tc::fence_before_sync();
      if (n + 1 < cnt) {
        ok = split(n + 1, 0) && warp_wait(bar(bMO1, n), par(n), abort_flag);   // S_n has been read
        if (ok) {
          if (tid == 128 && n + 2 < cnt) {
            load_wide(L::oQ, &tq, n + 2);
            nq = n + 3;
          }
          __syncwarp();
          if (mine) round_row(smem + L::oS, row, S);
          tc::fence_proxy_async();
          warp_arrive(bar(bState, n + 1));
        }
      }
    }
    if (ok && mine && a.hT && seg == sp.segments - 1)
      write_row(S, 1.f, a.hT + bh * st + static_cast<size_t>(row) * a.nv + 64 * slice);
    // no copy may outlive the CTA, whatever gave up (q and k of a chunk share a
    // barrier: a k left alone by an abort gets its q, so that it completes)
    if (tid == 128) {
      if (nq < nk) load_wide(L::oQ, &tq, nq);
      for (int n = max(0, nk - 2); n < nk; ++n) tc::mbar_wait(bar(bQK, n), par(n));
    }
    __syncwarp();
  } else if (warp < 12) {
    // ---------------------------------------------- read-out, one token per lane,
    // and the other half of V'
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o);
    int nv = 0;   // (tid 256) tiles requested
    if (tid == 256)
      for (; nv < min(2, cnt); ++nv) load_v(nv);
    __syncwarp();
    bool ok = split(0, 1);
    for (int n = 0; ok && n < cnt; ++n) {
      if (n + 1 < cnt) ok = warp_wait(bar(bMP, n), par(n), abort_flag) && split(n + 1, 1);
      ok = ok && warp_wait(bar(bMO1, n), par(n), abort_flag) &&
           warp_wait(bar(bMO2, n), par(n), abort_flag);
      if (!ok) break;
      if (tid == 256 && n + 2 < cnt) {   // v's readers, V'(n) and O2(n), are done
        load_v(n + 2);
        nv = n + 3;
      }
      __syncwarp();
      tc::fence_after_sync();
      const float f = a.scale * gates(n).head[row];
      warp_arrive(bar4(bGFree, n));
      const F2 ff = pack2(f, f), ss = pack2(a.scale, a.scale);
      const int t = n * kC + row;
      const bool live = t0 + t < t1;
      uint4* dst = reinterpret_cast<uint4*>(
          out + ((tok0 + t) * a.H + h) * static_cast<size_t>(a.nv) + 64 * slice);
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        float x[16], z[16];
        tc::tmem_ld16(tl + cO1 + (n & 1) * 64 + 16 * p, x);
        tc::tmem_ld16(tl + cA + (n & 1) * 128 + 64 + 16 * p, z);
        uint32_t y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = round2(fma2(ff, pack2(x[2 * i], x[2 * i + 1]),
                             mul2(ss, pack2(z[2 * i], z[2 * i + 1]))));
        if (live) {
          dst[2 * p] = make_uint4(y[0], y[1], y[2], y[3]);
          dst[2 * p + 1] = make_uint4(y[4], y[5], y[6], y[7]);
        }
      }
      tc::fence_before_sync();
      warp_arrive(bar(bFree, n));
    }
    if (tid == 256)
      for (int n = max(0, nv - 2); n < nv; ++n) tc::mbar_wait(bar(bV, n), par(n));
    __syncwarp();
  } else if (warp < 14) {
    // ---------------------------------------------- products, from two warps: one
    // warp's waits then pass while the other's products run
    const uint32_t go = lane == 0;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t idA = tc::idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t idO = tc::idesc_bf16(128, 64, 0, 1);
    constexpr uint32_t idP = tc::idesc_bf16(128, 128, 1, 1);
    // K-major tiles of 64-column blocks: the K step's byte offset
    auto kmaj = [](int k0) { return static_cast<uint64_t>((k0 >> 6) * kTile + (k0 & 63) * 2) >> 4; };
    auto rows = [](int k0) { return static_cast<uint64_t>(k0 * 128) >> 4; };
    uint32_t end = sb + L::oBar + 8 * bEnd;
    if (warp == 12) {
      const uint64_t dS = tc::smem_desc(sb + L::oS, 16, 1024);
      for (int n = 0; n < cnt; ++n) {
        if (!warp_wait(bar(bQK, n), par(n), abort_flag)) break;
        // the read-out of chunk n - 2 frees both accumulators
        if (n >= 2 && !warp_wait(bar(bFree, n), par(n - 2), abort_flag)) break;
        tc::fence_after_sync();
        const uint64_t dq = tc::smem_desc(sb + L::oQ + (n & 1) * L::kWide, 16, 1024);
        const uint64_t dk = tc::smem_desc(sb + L::oK + (n & 1) * L::kWide, 16, 1024);
#pragma unroll
        for (int k0 = 0; k0 < NK; k0 += 16)
          mma_if(go, tm + cA + (n & 1) * 128, dq + kmaj(k0), dk + kmaj(k0), idA, k0 > 0);
        commit_if(go, bar(bMA, n));
        if (!warp_wait(bar(bState, n), par(n), abort_flag)) break;
        tc::fence_after_sync();
#pragma unroll
        for (int k0 = 0; k0 < NK; k0 += 16)
          mma_if(go, tm + cO1 + (n & 1) * 64, dq + kmaj(k0), dS + rows(k0), idO, k0 > 0);
        commit_if(go, bar(bMO1, n));
      }
    } else {
      end += 8;
      const uint64_t dSplit = tc::smem_desc(sb + L::oSplit, kTile, 1024);
      for (int n = 0; n < cnt; ++n) {
        // the state has added the last P before it made its half of this V'
        if (!warp_wait(bar(bSplit, n), par(n), abort_flag) ||
            !warp_wait(bar(bQK, n), par(n), abort_flag))
          break;
        tc::fence_after_sync();
        const uint64_t dk = tc::smem_desc(sb + L::oK + (n & 1) * L::kWide, kTile, 1024);
#pragma unroll
        for (int k0 = 0; k0 < kC; k0 += 16)
          mma_if(go, tm + cP, dk + rows(k0), dSplit + rows(k0), idP, k0 > 0);
        commit_if(go, bar(bMP, n));
        if (!warp_wait(bar(bMask, n), par(n), abort_flag)) break;
        tc::fence_after_sync();
        const uint64_t dv = tc::smem_desc(sb + L::oV + (n & 1) * kTile, 16, 1024);
#pragma unroll
        for (int k0 = 0; k0 < kC; k0 += 16)
          mma_ta_if(go, tm + cA + (n & 1) * 128 + 64, tm + cA + (n & 1) * 128 + k0 / 2,
                    dv + rows(k0), idO, k0 > 0);
        commit_if(go, bar(bMO2, n));
      }
    }
    // nothing may still be reading shared memory when the CTA goes
    commit_if(go, end);
    tc::mbar_wait(end, 0);
  } else {
    // ---------------------------------------------- gates
    // the two warps take every other chunk, up to four chunks ahead of the readers
    float x[4], y[4];
    auto read = [&](float (&z)[4], int n) {
      read_gates(z, a, tok0 + n * kC, h, min(kC, t1 - t0 - n * kC));
    };
    const int first = warp - 14;
    if (first < cnt) read(x, first);
    for (int n = first; n < cnt; n += 2) {
      // the next values are on their way while these are used
      if (n + 2 < cnt) read(y, n + 2);
      const bool ok = n < 4 || warp_wait(bar4(bGFree, n), par4(n - 4), abort_flag);
      if (!ok) break;
      fill_gates(gates(n), x);
      warp_arrive(bar4(bGates, n));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = y[j];
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag) {
    // a bounded wait gave up: this CTA's results read NaN
    const float nan = __int_as_float(0x7fffffff);
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.o);
    for (int i = tid; i < (t1 - t0) * 64; i += kFwdThreads)
      out[((tok0 + i / 64) * a.H + h) * static_cast<size_t>(a.nv) + 64 * slice + i % 64] =
          __float2bfloat16_rn(nan);
    if (a.hT && seg == sp.segments - 1)
      for (int i = tid; i < NK * 64; i += kFwdThreads)
        a.hT[(static_cast<size_t>(bh) * NK + i / 64) * a.nv + 64 * slice + i % 64] = nan;
  }
  if (warp == 13) tc::tmem_dealloc(tmem, kCols);
}

// ------------------------------------------------------------------ states

// A segment's own end state, S = sum over its tokens of decay k v^T (REV: the
// gradient of its start state from its own read-outs, s sum of decay q dO^T,
// chunks in reverse), 64 value columns per CTA: the P product alone, V' double
// buffered so that a chunk is split while the previous one is multiplied.
constexpr int kStThreads = 224;   // 128: V' and state; loads; products; gates
constexpr int kStStages = 3;

enum : uint32_t { sFull = 0, sEmpty = 3, sSplit = 6, sP = 8, sGates = 10, sGFree = 12, sEnd = 14,
                  kStBars = 15 };

template <int NK>
struct StSmem {
  static constexpr uint32_t kWide = NK / 64 * kTile, kStage = kWide + kTile;
  static constexpr uint32_t oSplit = kStStages * kStage, oGates = oSplit + 4 * kTile,
                            oBar = oGates + 2 * sizeof(Gates), oSlot = oBar + 8 * kStBars + 4,
                            oAbort = oSlot + 4, bytes = oAbort + 8;
  static constexpr uint32_t launch = bytes + 1024;
};

template <int NK, bool REV>
__global__ void __launch_bounds__(kStThreads, 1)
    decay_states_tc(const DecayArgs a, const DecaySplit sp, const __grid_constant__ CUtensorMap tx,
                    const __grid_constant__ CUtensorMap ty) {
  using L = StSmem<NK>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = a.nv / 64, slice = blockIdx.x % slices;
  const int seg = blockIdx.x / slices + (REV ? 1 : 0);   // segment 0's gradient is not needed
  const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int t0 = seg * sp.seg_len, t1 = min(a.T, t0 + sp.seg_len);
  const int cnt = (t1 - t0 + kC - 1) / kC;
  auto at = [&](int n) { return t0 + (REV ? cnt - 1 - n : n) * kC; };
  auto bar = [&](uint32_t i) { return sb + L::oBar + 8 * i; };
  auto bar2 = [&](uint32_t i, int n) { return bar(i + (n & 1)); };
  auto par = [](int n) { return static_cast<uint32_t>(n >> 1) & 1u; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oAbort);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::oSlot);
  auto gates = [&](int n) -> Gates& {
    return *reinterpret_cast<Gates*>(smem + L::oGates + (n & 1) * sizeof(Gates));
  };
  if (warp == 5) tc::tmem_alloc(smem_u32(slot), 256);
  if (tid == 0) {
    for (uint32_t i = 0; i < kStBars; ++i)
      tc::mbar_init(bar(i), (i >= sSplit && i < sP) || (i >= sGFree && i < sEnd) ? 4 : 1);   // warps
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  const int row = 32 * (warp & 3) + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
  const bool mine = row < NK;
  const size_t st = static_cast<size_t>(NK) * a.nv;
  float* dst = (REV ? sp.D : sp.S) +
               (static_cast<size_t>(bh) * sp.slots + (REV ? seg : seg + 1)) * st + 64 * slice;

  if (warp < 4) {
    float S[64];
    read_row(S, nullptr);
    float prod = 1.f;
    auto split = [&](int n) {
      if (!warp_wait(bar2(sGates, n), par(n), abort_flag) ||
          !warp_wait(bar(sFull + n % kStStages), (n / kStStages) & 1, abort_flag))
        return false;
      const Gates& g = gates(n);
      split_row(smem + (n % kStStages) * L::kStage + L::kWide,
                smem + L::oSplit + (n & 1) * 2 * kTile, row, 0, REV ? g.head[row] : g.tail[row]);
      split_row(smem + (n % kStStages) * L::kStage + L::kWide,
                smem + L::oSplit + (n & 1) * 2 * kTile, row, 4, REV ? g.head[row] : g.tail[row]);
      tc::fence_proxy_async();
      warp_arrive(bar2(sSplit, n));
      return true;
    };
    bool ok = split(0);
    for (int n = 0; ok && n < cnt; ++n) {
      if (n + 1 < cnt) ok = split(n + 1);
      if (ok) ok = warp_wait(bar2(sP, n), par(n), abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const float all = gates(n).all;
      warp_arrive(bar2(sGFree, n));
      if (mine || NK == 128) add_state(S, all, tl + (n & 1) * 128);
      prod *= all;
      tc::fence_before_sync();
    }
    if (ok) {
      if (mine) write_row(S, REV ? a.scale : 1.f, dst + static_cast<size_t>(row) * a.nv);
      if (!REV && tid == 0 && slice == 0)
        sp.decay[static_cast<size_t>(bh) * sp.segments + seg] = prod;
    }
  } else if (warp == 4) {
    if (lane == 0) {
      int issued = 0;
      for (int n = 0; n < cnt; ++n) {
        const int s = n % kStStages;
        if (n >= kStStages && !wait(bar(sEmpty + s), (n / kStStages - 1) & 1, abort_flag)) break;
        tc::mbar_arrive_expect_tx(bar(sFull + s), L::kStage);
#pragma unroll
        for (int blk = 0; blk < NK / 64; ++blk)
          tc::tma_load_4d(sb + s * L::kStage + blk * kTile, &tx, 64 * blk, hk, at(n), b,
                          bar(sFull + s));
        tc::tma_load_4d(sb + s * L::kStage + L::kWide, &ty, 64 * slice, h, at(n), b,
                        bar(sFull + s));
        issued = n + 1;
      }
      for (int n = max(0, issued - kStStages); n < issued; ++n)
        tc::mbar_wait(bar(sFull + n % kStStages), (n / kStStages) & 1);
    }
  } else if (warp == 5) {
    const uint32_t go = lane == 0;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t idP = tc::idesc_bf16(128, 128, 1, 1);
    for (int n = 0; n < cnt; ++n) {
      // (the state has read this accumulator, chunk n - 2's, before it made this V')
      if (!warp_wait(bar2(sSplit, n), par(n), abort_flag)) break;
      tc::fence_after_sync();
      const uint64_t dx = tc::smem_desc(sb + (n % kStStages) * L::kStage, kTile, 1024);
      const uint64_t dy = tc::smem_desc(sb + L::oSplit + (n & 1) * 2 * kTile, kTile, 1024);
#pragma unroll
      for (int k0 = 0; k0 < kC; k0 += 16)
        mma_if(go, tm + (n & 1) * 128, dx + ((k0 * 128) >> 4), dy + ((k0 * 128) >> 4), idP, k0 > 0);
      commit_if(go, bar2(sP, n));
      commit_if(go, bar(sEmpty + n % kStStages));
    }
    commit_if(go, bar(sEnd));
    tc::mbar_wait(bar(sEnd), 0);
  } else {
    float x[4], y[4];
    auto read = [&](float (&z)[4], int n) {
      read_gates(z, a, static_cast<size_t>(b) * a.T + at(n), h, min(kC, t1 - at(n)));
    };
    read(x, 0);
    for (int n = 0; n < cnt; ++n) {
      if (n + 1 < cnt) read(y, n + 1);
      const bool ok = n < 2 || warp_wait(bar2(sGFree, n), par(n - 2), abort_flag);
      if (!ok) break;
      fill_gates(gates(n), x);
      warp_arrive(bar2(sGates, n));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = y[j];
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag)   // a bounded wait gave up: the state, and all that follows, reads NaN
    for (int i = tid; i < NK * 64; i += kStThreads)
      dst[static_cast<size_t>(i / 64) * a.nv + i % 64] = __int_as_float(0x7fffffff);
  if (warp == 5) tc::tmem_dealloc(tmem, 256);
}

template <class Kern>
cudaError_t opt_in(Kern kern, uint32_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes));
}

template <int NK>
cudaError_t fwd(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  using L = FwdSmem<NK>;
  static_assert(L::launch <= 232448, "shared memory budget of one CTA");
  CUtensorMap tq, tk, tv;
  if (!make_rows_tmap(&tq, a.q, a.B, a.T, a.Hk, NK, a.sq) ||
      !make_rows_tmap(&tk, a.k, a.B, a.T, a.Hk, NK, a.sk) ||
      !make_rows_tmap(&tv, a.v, a.B, a.T, a.H, a.nv, a.sv))
    return cudaErrorInvalidValue;
  const cudaError_t err = opt_in(decay_fwd_tc<NK>, L::launch);
  if (err != cudaSuccess) return err;
  decay_fwd_tc<NK><<<dim3(sp.segments * (a.nv / 64), a.B * a.H), kFwdThreads, L::launch, stream>>>(
      a, sp, tq, tk, tv);
  return cudaGetLastError();
}

template <int NK, bool REV>
cudaError_t states(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  using L = StSmem<NK>;
  static_assert(L::launch <= 232448, "shared memory budget of one CTA");
  const long long so = static_cast<long long>(a.H) * a.nv;
  CUtensorMap tx, ty;
  if (!make_rows_tmap(&tx, REV ? a.q : a.k, a.B, a.T, a.Hk, NK, REV ? a.sq : a.sk) ||
      !make_rows_tmap(&ty, REV ? a.dO : a.v, a.B, a.T, a.H, a.nv, REV ? so : a.sv))
    return cudaErrorInvalidValue;
  const cudaError_t err = opt_in(decay_states_tc<NK, REV>, L::launch);
  if (err != cudaSuccess) return err;
  const int segs = REV ? sp.segments - 1 : sp.slots - 1;
  decay_states_tc<NK, REV><<<dim3(segs * (a.nv / 64), a.B * a.H), kStThreads, L::launch, stream>>>(
      a, sp, tx, ty);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_fwd_tc(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  return a.nk == 64 ? fwd<64>(a, sp, stream) : fwd<128>(a, sp, stream);
}
cudaError_t launch_decay_states_tc(const DecayArgs& a, const DecaySplit& sp, bool reverse,
                                   cudaStream_t stream) {
  if ((reverse ? sp.segments : sp.slots) < 2) return cudaSuccess;
  if (reverse)
    return a.nk == 64 ? states<64, true>(a, sp, stream) : states<128, true>(a, sp, stream);
  return a.nk == 64 ? states<64, false>(a, sp, stream) : states<128, false>(a, sp, stream);
}

}  // namespace gdr
