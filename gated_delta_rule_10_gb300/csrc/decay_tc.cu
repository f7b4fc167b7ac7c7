// Linear attention with a decay for each head, chunked, for bf16 inputs on
// tcgen05: the forward, its three gradients and the segments' own states.
//
// One walk over a sequence serves all four results. It reads rows x_t, y_t of W
// channels and z_t of 64 (a column slice of the third tensor), carries a state R
// (W x 64, fp32) and writes, for every token t,
//   out_t = f_t R^T x_t + s sum_i D_ti (x_t . y_i) z_i,
// over the tokens i <= t of its chunk of 128, with D the decay between two tokens
// and f_t = s e^{G_t}; after the chunk, R = e^{G_C} R + sum_i e^{G_C-G_i} y_i z_i^T.
//   forward   x, y, z = q, k, v     R = S     out = o
//   dq        x, y, z = dO, v, k    R = S^T   out = dq
// Backward (REV) the chunks are taken from the end, i >= t, f_t = e^{G_C-G_t}, and
// R = e^{G_C} R + s sum_i e^{G_i} y_i z_i^T:
//   dv        x, y, z = k, q, dO    R = D     out = dv     (D: the gradient of S)
//   dk        x, y, z = v, dO, q    R = D^T   out = dk
//
// Four products a chunk:
//   A  = X Y^T                        (128 x 128, K = W)
//   O1 = X R                          (128 x 64,  K = W)
//   O2 = (A . D) Z                    (128 x 64,  K = 128, A . D from tensor memory)
//   P  = Y^T Z'                       (W x 64,    K = 128), Z' the decayed Z.
// x, y and z go from TMA to the tensor cores as they are. A . D and the R of the
// read-out are rounded to bf16 (the result is rounded to bf16 anyway); the decayed
// Z' is split into two bf16 terms, side by side in one N = 128 product, because it
// enters the fp32 state, whose error would otherwise be bf16's (1.7e-3; with two
// terms 2.4e-6 of 64 bits). A third term would leave 1e-7 of hT and dh0; in this form of
// the walk the forward of 4 x 4096 x 16 x 128 takes 87 us instead of 68 with one for half
// of the tokens alone, for which there is room.
//
// FINE (dq and dk): the gate's gradient needs f_t (R^T x_t) . p_t in fp32, p the
// partner row (q or k), and sums of those differences over thousands of tokens. Two
// terms are not enough there (2e-5 of a fixed decay's gradient at 1100 tokens): Z'
// and, for O1, R take three each, which is all of fp32 (states 1e-7, gradient 1e-6).
// A chunk then takes ~7000 cycles, against ~4000: shared memory has room for one tile
// of z and Z' of 64 tokens at a time, so Z' is made by the mask's threads from rows of z
// read ahead into registers (the state's threads, who round R meanwhile, were what the
// rest waited for), the first term of R and the others sit side by side in one N = 128
// product, and the result leaves through z's tile (396 -> 368 us for all gradients of
// 4 x 4096 x 16 x 128).
//
// Only R_{n+1} <- R_n is a chain, and it holds no product: P of any chunk can be
// ready before R is. A and O1 are issued by one warp, P and O2 by another: the
// issue of a product takes as long as the product (~52 cycles at any of these
// shapes), and the waits of one warp pass while the other's products run (58 ->
// 40 us for the products of 4 x 4096 x 16 x 128 alone). Each tile is loaded
// again as soon as its last reader is done, about one chunk's time ahead.
// The two column halves of a head re-read x and y (from L2) and repeat A.
// Forward of 4 x 4096 x 16 x 128: 68 us, 0.6 of measured HBM bandwidth; 1 x 65536 x 32 x
// 128: 675 us with the states. No unit is near its rate there: of the busiest SM the
// load/store pipe to shared memory is 0.45 busy, issue slots 0.48, tensor pipe 0.31 over
// all SMs, DRAM 0.47; 24 of 152 SMs have no CTA. The ~4000 cycles of a chunk go to the
// waits along its chains of roles, each a hand-over through an mbarrier and a read of
// tensor or shared memory: of 8.2 warp cycles an instruction 2.9 are such waits, 1.3
// fixed latencies and 0.8 instruction fetch (0.83 of the fetches hit).
#include <algorithm>

#include "decay_tc.cuh"
#include "tma.h"

namespace gdr {
namespace {

using namespace dtc;

// ------------------------------------------------------------------ walk

struct Walk {
  int x_heads, y_heads, z_heads;   // heads of each tensor: H or Hk
  int nz;                          // width of z and of the result
  void* out;                       // [B, T, H, nz] bf16, or
  float* part;                     // the same in fp32 (a head's part of a shared gradient)
  const float* start;              // first state; null: zero
  size_t start_bh;                 // its elements between (batch, head)s
  bool chained;                    // it is the slot of this segment's edge
  int row_step, col_step;          // its elements between rows (W) and columns (z)
  float* end;                      // last state [B * H, W, nz], or null
  const __nv_bfloat16 *z, *partner;   // FINE: z itself, and the rows whose dot product with
  long long z_stride, partner_stride;   // the result is wanted
  float* flow;                     // [slices, B * H, T], that product
};

constexpr int kThreads = 512;   // 3 x 128: mask, state, read-out; products (2); gates; loads
constexpr uint32_t kCols = 512;

// Tensor-memory columns of chunk n: two buffers of A, whose columns 0..63 take
// A . D as bf16 and 64..127 O2 once A has been read, two of O1 (FINE: one, with 64
// columns for the first term of R and 64 for the others), and P.
template <bool FINE>
struct Cols {
  __device__ static uint32_t A(int n) { return (n & 1) * 128; }
  __device__ static uint32_t O2(int n) { return A(n) + 64; }
  __device__ static uint32_t O1(int n) { return 256 + (FINE ? 0 : (n & 1) * 64); }
  static constexpr uint32_t P = 384;
};

enum : uint32_t {   // mbarriers, each a pair for even and odd chunks
  bXY = 0, bZ = 2,                           // tiles landed
  bMA = 4, bMO1 = 6, bMO2 = 8, bMP = 10,     // products complete
  bMask = 12, bState = 16, bFree = 18,
  bSplit = 14,                               // (FINE: Z' of tokens 0..63 and 64..127)
  bGates = 20, bGFree = 24,                  // a ring of four (FINE: two) chunks' gates
  bEnd = 28, bMP0 = 30,                      // (P of tokens 0..63 complete)
  bAdd = 32,                                 // (FINE: P read)
  kBars = 34
};

constexpr uint32_t kHalf = kTile / 2;   // 64 rows of 64 bf16 columns

template <int W, bool FINE>
struct WalkSmem {
  static constexpr uint32_t kWide = W / 64 * kTile, kZ = FINE ? 1 : 2, kRing = FINE ? 2 : 4;
  static constexpr uint32_t oX = 0, oY = oX + 2 * kWide, oZ = oY + 2 * kWide,
                            oSplit = oZ + kZ * kTile, oR = oSplit + (FINE ? 3 * kHalf : 2 * kTile),
                            kR = W * 128, oGates = oR + (FINE ? 3 : 1) * kR,
                            oBar = oGates + kRing * sizeof(Gates), oSlot = oBar + 8 * kBars,
                            oAbort = oSlot + 4, bytes = oAbort + 12;
  static constexpr uint32_t launch = bytes + 1024;   // room to align the base
};

// One CTA's walk over segment `seg` of (batch, head) `bh`, columns 64 slice .. + 63.
template <int W, bool REV, bool FINE>
__device__ __forceinline__ void walk_cta(const DecayArgs& a, const DecaySplit& sp, const Walk& w,
                                         const CUtensorMap* tx, const CUtensorMap* ty,
                                         const CUtensorMap* tz, const CUtensorMap* tout, int seg,
                                         int slice, int bh) {
  using L = WalkSmem<W, FINE>;
  using C = Cols<FINE>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = bh / a.H, h = bh % a.H;
  const int t0 = seg * sp.seg_len, t1 = min(a.T, t0 + sp.seg_len);
  const int cnt = (t1 - t0 + kC - 1) / kC;
  const size_t tok = static_cast<size_t>(b) * a.T;
  auto at = [&](int n) { return t0 + (REV ? cnt - 1 - n : n) * kC; };   // chunk n's first token
  auto bar = [&](uint32_t i, int n) { return sb + L::oBar + 8 * (i + (n & 1)); };
  auto par = [](int n) { return static_cast<uint32_t>(n >> 1) & 1u; };
  constexpr int kRing = L::kRing;
  auto bar4 = [&](uint32_t i, int n) { return sb + L::oBar + 8 * (i + (n & (kRing - 1))); };
  auto par4 = [](int n) { return static_cast<uint32_t>(n / kRing) & 1u; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oAbort);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::oSlot);
  auto gates = [&](int n) -> Gates& {
    return *reinterpret_cast<Gates*>(smem + L::oGates + (n & (kRing - 1)) * sizeof(Gates));
  };
  auto zslot = [](int n) { return FINE ? 0u : static_cast<uint32_t>(n & 1) * kTile; };
  if (warp == 13) tc::tmem_alloc(smem_u32(slot), kCols);
  if (tid == 0) {
    for (uint32_t i = 0; i < kBars; ++i) {
      uint32_t count = i < bZ ? 2 : 1;   // x and y land on one barrier
      if (i >= bMask && i < bGates) count = !FINE && (i == bSplit || i == bSplit + 1) ? 8 : 4;   // warps
      if (i >= bGFree && i < bEnd) count = 8;
      if (i >= bAdd) count = 4;
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

  // tiles of chunk n into their slots (one lane of the loading warp)
  auto load_wide = [&](uint32_t base, const CUtensorMap* m, int heads, int n) {
    tc::mbar_arrive_expect_tx(bar(bXY, n), L::kWide);
#pragma unroll
    for (int blk = 0; blk < W / 64; ++blk)
      tc::tma_load_4d(sb + base + (n & 1) * L::kWide + blk * kTile, m, 64 * blk,
                      h / (a.H / heads), at(n), b, bar(bXY, n));
  };
  auto load_x = [&](int n) { load_wide(L::oX, tx, w.x_heads, n); };
  auto load_y = [&](int n) { load_wide(L::oY, ty, w.y_heads, n); };
  auto load_z = [&](int n) {
    tc::mbar_arrive_expect_tx(bar(bZ, n), kTile);
    tc::tma_load_4d(sb + L::oZ + zslot(n), tz, 64 * slice, h / (a.H / w.z_heads), at(n), b,
                    bar(bZ, n));
  };
  // Z' by the state's and the read-out's 256 threads, half the columns of this lane's
  // token each, the caller having waited for P(n - 1), its last reader.
  auto split = [&](int n, int half) {
    if (!warp_wait(bar4(bGates, n), par4(n), abort_flag) ||
        !warp_wait(bar(bZ, n), par(n), abort_flag))
      return false;
    const Gates& g = gates(n);
    const float f = REV ? a.scale * g.head[row] : g.tail[row];
#pragma unroll 1
    for (int c = 4 * half; c < 4 * half + 4; c += 2)
      split_row<2>(sb + L::oZ + zslot(n), sb + L::oSplit, kTile, row, c, f);
    tc::fence_proxy_async();
    warp_arrive(bar(bSplit, n));
    return true;
  };
  // FINE: by the mask's threads, tokens 64 half .. + 63, a quarter of a row at a time, from
  // registers that were filled a half ahead (through the one z tile Z' would wait for the
  // O2 before and a load).
  uint4 zr[2][2];
  auto fetch = [&](int n, int half, int set) {
    const int t = at(n) + 64 * half + 32 * set + (tid >> 2);
    const uint4* p = reinterpret_cast<const uint4*>(
        w.z + static_cast<long long>(tok + t) * w.z_stride + (h / (a.H / w.z_heads)) * w.nz +
        64 * slice + 16 * (tid & 3));
#pragma unroll
    for (int i = 0; i < 2; ++i)
      zr[set][i] = n < cnt && t < t1 ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
  };
  auto split_half = [&](int n, int half) {
    if (half == 0) {
      if (!warp_wait(bar4(bGates, n), par4(n), abort_flag) ||
          (n > 0 && !warp_wait(bar(bMP, n - 1), par(n - 1), abort_flag)))
        return false;
    } else if (!warp_wait(sb + L::oBar + 8 * (bMP0 + (n & 1)), par(n), abort_flag)) {
      return false;
    }
    const Gates& g = gates(n);
#pragma unroll
    for (int set = 0; set < 2; ++set) {
      const int to = 32 * set + (tid >> 2), r = 64 * half + to;
      split_pair<3>(zr[set], sb + L::oSplit, kHalf, to, 2 * (tid & 3),
                    REV ? a.scale * g.head[r] : g.tail[r]);
      fetch(n + half, half ^ 1, set);
    }
    tc::fence_proxy_async();
    warp_arrive(sb + L::oBar + 8 * (bSplit + half));
    return true;
  };

  if (warp < 4) {
    // ---------------------------------------------- A . D, one token per lane
    if (FINE) {
      fetch(0, 0, 0);
      fetch(0, 0, 1);
    }
    for (int n = 0; n < cnt; ++n) {
      bool ok = warp_wait(bar4(bGates, n), par4(n), abort_flag) &&
                warp_wait(bar(bMA, n), par(n), abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const Gates& g = gates(n);
      const float lr = g.loc[row];
      const uint32_t allow = g.allow[row];
#pragma unroll 1
      for (int cb = 0; cb < 4; ++cb) {
        uint32_t r[16];
        if (REV ? cb < quad : cb > quad) {
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = 0u;
        } else {
          float x[32];
          tc::tmem_ld32(tl + C::A(n) + 32 * cb, x);
          if (cb == quad) {
            const float* f = g.loc + 32 * cb;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 v = *reinterpret_cast<const float4*>(f + i);
              const float c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float e = exp2_fast(REV ? c[j] - lr : lr - c[j]);
                x[i + j] = (allow >> (i + j)) & 1u ? x[i + j] * e : 0.f;
              }
              r[i / 2] = pack_bf16x2(x[i], x[i + 1]);
              r[i / 2 + 1] = pack_bf16x2(x[i + 2], x[i + 3]);
            }
          } else {
            // forward: row[t] col[i]; backward: col[t] of this block pair, row[i]
            const float fr = REV ? g.col[col_at(cb) + row] : g.row[row];
            const float* f = REV ? g.row + 32 * cb : g.col + col_at(quad) + 32 * cb;
            const F2 ff = pack2(fr, fr);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(f + i);
              r[i / 2] = round2(mul2(pack2(x[i], x[i + 1]), mul2(ff, c.x)));
              r[i / 2 + 1] = round2(mul2(pack2(x[i + 2], x[i + 3]), mul2(ff, c.y)));
            }
          }
        }
        tc::tmem_st16(tl + C::A(n) + 16 * cb, r);   // over columns already read
      }
      tc::tmem_st_wait();
      tc::fence_before_sync();
      warp_arrive(bar(bMask, n));
      if (FINE) {
#pragma unroll 1
        for (int half = 0; ok && half < 2; ++half) ok = split_half(n, half);
        if (!ok) break;
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------- the state, one row per lane, and
    // half of Z'
    const bool mine = row < W;
    float R[64];
    const size_t edge = w.chained ? sp.slot_of(REV ? seg + 1 : seg) : 0;
    read_row(R, w.start && mine ? w.start + bh * w.start_bh + edge * W * w.nz +
                                      static_cast<size_t>(row) * w.row_step +
                                      static_cast<size_t>(64 * slice) * w.col_step
                                : nullptr,
             w.col_step);
    bool ok = true;
    auto publish = [&](int n) {   // R as an operand of O1(n)
      if (mine) round_row<FINE>(sb + L::oR, L::kR, row, R);
      tc::fence_proxy_async();
      warp_arrive(bar(bState, n));
    };
    auto add = [&](int n) {
      if (!warp_wait(bar(bMP, n), par(n), abort_flag)) return false;
      tc::fence_after_sync();
      const float all = gates(n).all;
      warp_arrive(bar4(bGFree, n));
      if (mine || W == 128) add_state(R, all, tl + C::P);
      tc::fence_before_sync();
      if (FINE) warp_arrive(bar(bAdd, n));
      return true;
    };
    // (one copy of each step in the loops: the roles' code together is more than the
    // instruction cache holds as it is)
    if constexpr (FINE) {
#pragma unroll 1
      for (int n = 0; ok && n < cnt; ++n) {
        if (n > 0) ok = warp_wait(bar(bMO1, n - 1), par(n - 1), abort_flag);   // has read R
        if (!ok) break;
        publish(n);
        ok = add(n);
      }
    } else {
      publish(0);
      ok = split(0, 0);
      for (int n = 0; ok && n < cnt; ++n) {
        ok = add(n);
        if (!ok || n + 1 == cnt) break;
        ok = split(n + 1, 0) && warp_wait(bar(bMO1, n), par(n), abort_flag);   // R_n has been read
        if (ok) publish(n + 1);
      }
    }
    if (ok && mine && w.end && seg == (REV ? 0 : sp.segments - 1))
      write_row(R, 1.f, w.end + (static_cast<size_t>(bh) * W + row) * w.nz + 64 * slice);
    if constexpr (FINE && REV) {
      // <h0, D> where the gate's gradient starts, from three terms (dh0 has two)
      if (ok && mine && a.h0 && seg == 0) {
        const float* s = a.h0 + (static_cast<size_t>(bh) * w.nz + 64 * slice) * W + row;
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < 64; ++j) dot = fmaf(R[j], s[j * W], dot);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
        if (lane == 0) sp.first[bh * sp.firsts + slice * (W / 32) + quad] = dot;
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------- read-out, one token per lane, and
    // the other half of Z'
    bool ok = true;
    if (!FINE) ok = split(0, 1);
    for (int n = 0; ok && n < cnt; ++n) {
      const int t = at(n) + row;
      const bool live = t < t1;
      uint4 pr[FINE ? 8 : 1];
      if (FINE) {   // the partner's row, on its way while the products run
        const uint4* p = reinterpret_cast<const uint4*>(
            w.partner + static_cast<long long>(tok + t) * w.partner_stride +
            (h / (a.H / w.z_heads)) * w.nz + 64 * slice);
#pragma unroll
        for (int i = 0; i < 8; ++i) pr[i] = live ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
      } else if (n + 1 < cnt) {
        ok = warp_wait(bar(bMP, n), par(n), abort_flag) && split(n + 1, 1);
      }
      ok = ok && warp_wait(bar(bMO1, n), par(n), abort_flag) &&
           warp_wait(bar(bMO2, n), par(n), abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const float f = REV ? gates(n).tail[row] : a.scale * gates(n).head[row];
      warp_arrive(bar4(bGFree, n));
      const F2 ff = pack2(f, f), ss = pack2(a.scale, a.scale);
      const size_t to = ((tok + t) * a.H + h) * static_cast<size_t>(w.nz) + 64 * slice;
      // FINE: the row goes out through z's tile, which O2 has read last. Else it is stored
      // from here, two lanes on 32 bytes of one row: what two rows' lanes hold is
      // exchanged first (16 bytes to each of 32 rows take the SM twice as long, and z's or
      // x's tile is asked for too soon to wait for a store: 70 -> 81 us)
      const uint32_t tile = sb + L::oZ + row * 128;
      const uint32_t odd = lane & 1;
      const size_t pitch = static_cast<size_t>(a.H) * w.nz;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(w.out) + to - (odd ? pitch : 0) + 8 * odd;
      const bool live0 = t - static_cast<int>(odd) < t1, live1 = t + 1 - static_cast<int>(odd) < t1;
      F2 dot = pack2(0.f, 0.f);
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        float x[16], z[16];
        if (FINE) {
          tmem_ld16x2(tl + C::O1(n) + 16 * p, tl + C::O1(n) + 64 + 16 * p, x, z);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] += z[i];
          tc::tmem_ld16(tl + C::O2(n) + 16 * p, z);
        } else {
          tmem_ld16x2(tl + C::O1(n) + 16 * p, tl + C::O2(n) + 16 * p, x, z);
        }
        F2 y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = fma2(ff, pack2(x[2 * i], x[2 * i + 1]),
                      mul2(ss, pack2(z[2 * i], z[2 * i + 1])));
        if (FINE) {
          const uint32_t v[8] = {pr[0].x, pr[0].y, pr[0].z, pr[0].w,
                                 pr[1].x, pr[1].y, pr[1].z, pr[1].w};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dot = fma2(pack2(x[2 * i], x[2 * i + 1]), widen2(v[i]), dot);
#pragma unroll
          for (int i = 0; i < 6; ++i) pr[i] = pr[i + 2];   // (the loop stays rolled)
          if (w.part) {
            if (live) {
              ulonglong2* d = reinterpret_cast<ulonglong2*>(w.part + to + 16 * p);
#pragma unroll
              for (int i = 0; i < 4; ++i) d[i] = make_ulonglong2(y[2 * i], y[2 * i + 1]);
            }
            continue;
          }
        }
        uint32_t u[2][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i >> 2][i & 3] = round2(y[i]);
        if (FINE) {
#pragma unroll
          for (int i = 0; i < 2; ++i) sts4(tile + (((2 * p + i) ^ (row & 7)) << 4), u[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? u[0][i] : u[1][i], 1);
            u[0][i] = odd ? other : u[0][i];
            u[1][i] = odd ? u[1][i] : other;
          }
          if (live0)
            *reinterpret_cast<uint4*>(dst + 16 * p) =
                make_uint4(u[0][0], u[0][1], u[0][2], u[0][3]);
          if (live1)
            *reinterpret_cast<uint4*>(dst + pitch + 16 * p) =
                make_uint4(u[1][0], u[1][1], u[1][2], u[1][3]);
        }
      }
      if (FINE) {
        float d0, d1;
        unpack2(dot, d0, d1);
        if (live)
          w.flow[(static_cast<size_t>(slice) * a.B * a.H + bh) * a.T + t] = f * (d0 + d1);
      }
      if (FINE) tc::fence_proxy_async();
      tc::fence_before_sync();
      warp_arrive(bar(bFree, n));
    }
  } else if (warp < 14) {
    // ---------------------------------------------- products
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
      const uint64_t dR = tc::smem_desc(sb + L::oR, FINE ? L::kR : 16, 1024);
      const uint64_t dR3 = tc::smem_desc(sb + L::oR + 2 * L::kR, 16, 1024);
      constexpr uint32_t idR = tc::idesc_bf16(128, FINE ? 128 : 64, 0, 1);
      auto products_a = [&](int n) {
        if (!warp_wait(bar(bXY, n), par(n), abort_flag)) return false;
        tc::fence_after_sync();
        const uint64_t dx = tc::smem_desc(sb + L::oX + (n & 1) * L::kWide, 16, 1024);
        const uint64_t dy = tc::smem_desc(sb + L::oY + (n & 1) * L::kWide, 16, 1024);
#pragma unroll 1
        for (int k0 = 0; k0 < W; k0 += 16)
          mma_if(go, tm + C::A(n), dx + kmaj(k0), dy + kmaj(k0), idA, k0 > 0);
        commit_if(go, bar(bMA, n));
        return true;
      };
      for (int n = FINE ? -1 : 0; n < cnt; ++n) {
        // the read-out frees the buffers of A and O1: of chunk n - 2 for this one's, or
        // (FINE, the one buffer of O1 and the next chunk's A, which the longer way
        // through the mask to Z' waits for) of chunk n - 1
        const int freed = FINE ? n - 1 : n - 2;
        if (freed >= 0 && !warp_wait(bar(bFree, freed), par(freed), abort_flag)) break;
        if (FINE) {
          if (n + 1 < cnt && !products_a(n + 1)) break;
          if (n < 0) continue;
        } else if (!products_a(n)) {
          break;
        }
        if (!warp_wait(bar(bState, n), par(n), abort_flag)) break;
        tc::fence_after_sync();
        const uint64_t dx = tc::smem_desc(sb + L::oX + (n & 1) * L::kWide, 16, 1024);
#pragma unroll 1
        for (int k0 = 0; k0 < W; k0 += 16) {
          mma_if(go, tm + C::O1(n), dx + kmaj(k0), dR + rows(k0), idR, k0 > 0);
          if (FINE) mma_if(go, tm + C::O1(n) + 64, dx + kmaj(k0), dR3 + rows(k0), idO, 1);
        }
        commit_if(go, bar(bMO1, n));
      }
    } else {
      end += 8;
      const uint64_t dSplit = tc::smem_desc(sb + L::oSplit, FINE ? kHalf : kTile, 1024);
      const uint64_t dThird = tc::smem_desc(sb + L::oSplit + 2 * kHalf, 16, 1024);
      constexpr uint32_t idT = tc::idesc_bf16(128, 64, 1, 1);
      for (int n = 0; n < cnt; ++n) {
        if (!warp_wait(bar(bXY, n), par(n), abort_flag)) break;
        const uint64_t dy = tc::smem_desc(sb + L::oY + (n & 1) * L::kWide, kTile, 1024);
        // (the state has added the last P before it made its part of this Z')
        if constexpr (FINE) {
          bool ok = true;
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            ok = warp_wait(sb + L::oBar + 8 * (bSplit + half), n & 1, abort_flag);
            if (ok && half == 0 && n > 0) ok = warp_wait(bar(bAdd, n - 1), par(n - 1), abort_flag);
            if (!ok) break;
            tc::fence_after_sync();
#pragma unroll 1
            for (int k0 = 0; k0 < 64; k0 += 16) {
              const uint64_t y = dy + rows(64 * half + k0);
              mma_if(go, tm + C::P, y, dSplit + rows(k0), idP, half + k0 > 0);
              mma_if(go, tm + C::P + 64, y, dThird + rows(k0), idT, 1);
            }
            commit_if(go, half ? bar(bMP, n) : sb + L::oBar + 8 * (bMP0 + (n & 1)));
          }
          if (!ok) break;
        } else {
          if (!warp_wait(bar(bSplit, n), par(n), abort_flag)) break;
          tc::fence_after_sync();
#pragma unroll 1
          for (int k0 = 0; k0 < kC; k0 += 16)
            mma_if(go, tm + C::P, dy + rows(k0), dSplit + rows(k0), idP, k0 > 0);
          commit_if(go, bar(bMP, n));
        }
        if (!warp_wait(bar(bMask, n), par(n), abort_flag)) break;
        tc::fence_after_sync();
        if (FINE && !warp_wait(bar(bZ, n), par(n), abort_flag)) break;
        const uint64_t dz = tc::smem_desc(sb + L::oZ + zslot(n), 16, 1024);
#pragma unroll 1
        for (int k0 = 0; k0 < kC; k0 += 16)
          mma_ta_if(go, tm + C::O2(n), tm + C::A(n) + k0 / 2, dz + rows(k0), idO, k0 > 0);
        commit_if(go, bar(bMO2, n));
      }
    }
    // nothing may still be reading shared memory when the CTA goes
    commit_if(go, end);
    tc::mbar_wait(end, 0);
  } else if (warp == 15) {
    // ---------------------------------------------- loads: a slot is free once the last
    // product that reads it is complete, seen here at once (left to the roles, a z
    // tile was asked for a third of a chunk later and waited for)
    if (lane == 0) {
      constexpr int kAhead = FINE ? 1 : 2;   // z tiles
      int nx = 0, ny = 0, nz = 0;   // tiles requested
      for (; nx < min(2, cnt); ++nx, ++ny) {
        load_x(nx);
        load_y(ny);
      }
      for (; nz < min(kAhead, cnt); ++nz) load_z(nz);
      for (int n = 0; n < cnt; ++n) {
        if (n + 2 < cnt) {
          if (!wait(bar(bMO1, n), par(n), abort_flag)) break;   // (its warp issued A first)
          load_x(nx++);
          if (!wait(bar(bMP, n), par(n), abort_flag) || !wait(bar(bMA, n), par(n), abort_flag)) break;
          load_y(ny++);
        }
        if (FINE) {
          // z's tile holds the result now; tokens past the sequence's end are not written
          if (!wait(bar(bFree, n), par(n), abort_flag)) break;
          if (!w.part) {
            tc::tma_store_4d(tout, 64 * slice, h, at(n), b, sb + L::oZ);
            tc::bulk_commit();
            tc::bulk_wait_read<0>();
          }
        } else if (n + 2 < cnt) {
          // O2(n) follows P(n), which waited for Z'(n): z's readers are done
          if (!wait(bar(bMO2, n), par(n), abort_flag)) break;
        }
        if (n + kAhead < cnt) load_z(nz++);
      }
      if (FINE) tc::bulk_wait_all<0>();
      // no copy may outlive the CTA, whatever gave up (x and y of a chunk share a
      // barrier: an x left alone by an abort gets its y, so that it completes)
      if (ny < nx) load_y(ny);
      for (int n = max(0, nx - 2); n < nx; ++n) tc::mbar_wait(bar(bXY, n), par(n));
      for (int n = max(0, nz - kAhead); n < nz; ++n) tc::mbar_wait(bar(bZ, n), par(n));
    }
  } else {
    // ---------------------------------------------- gates, up to a ring ahead of the
    // readers
    float x[4], y[4];
    auto read = [&](float (&v)[4], int n) {
      read_gates(v, a, tok + at(n), h, min(kC, t1 - at(n)));
    };
    read(x, 0);
    for (int n = 0; n < cnt; ++n) {
      // the next values are on their way while these are used
      if (n + 1 < cnt) read(y, n + 1);
      if (n >= kRing && !warp_wait(bar4(bGFree, n), par4(n - kRing), abort_flag)) break;
      fill_gates<REV>(gates(n), x);
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
    for (int i = tid; i < (t1 - t0) * 64; i += kThreads) {
      const size_t to = ((tok + t0 + i / 64) * a.H + h) * static_cast<size_t>(w.nz) + 64 * slice +
                        i % 64;
      if (w.part) w.part[to] = nan;
      else static_cast<__nv_bfloat16*>(w.out)[to] = __float2bfloat16_rn(nan);
    }
    if (FINE)
      for (int i = tid; i < t1 - t0; i += kThreads)
        w.flow[(static_cast<size_t>(slice) * a.B * a.H + bh) * a.T + t0 + i] = nan;
    if (w.end && seg == (REV ? 0 : sp.segments - 1))
      for (int i = tid; i < W * 64; i += kThreads)
        w.end[(static_cast<size_t>(bh) * W + i / 64) * w.nz + 64 * slice + i % 64] = nan;
  }
  if (warp == 13) tc::tmem_dealloc(tmem, kCols);
}

template <int W>
__global__ void __launch_bounds__(kThreads, 1)
    decay_fwd_tc(const DecayArgs a, const DecaySplit sp, const Walk w,
                 const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap ty,
                 const __grid_constant__ CUtensorMap tz) {
  const int slices = w.nz / 64;
  walk_cta<W, false, false>(a, sp, w, &tx, &ty, &tz, nullptr, blockIdx.x / slices, blockIdx.x % slices,
                            blockIdx.y);
}

// ------------------------------------------------------------------ states

// A piece's own end state, S = sum over its tokens of decay k v^T (REV: the
// gradient of its start state from its own read-outs, s sum of decay q dO^T,
// chunks in reverse), 64 value columns per CTA: the P product alone, V' (whole chunks)
// double buffered so that a chunk is split while the previous one is multiplied. 180 us
// for the first half of 1 x 65536 x 32 x 128 (537 MB, 79 at the measured bandwidth), 22 us
// for 18 of 19 pieces of 1 x 29999 x 4 x 128; a third term costs a tenth more. Each chunk
// waits for its V' to be read, split and written back before its product, and the state
// for that.
constexpr int kStThreads = 352;   // 128: half of V' and state; 128: the other half; loads;
                                  // products; gates
constexpr int kStStages = 2;

enum : uint32_t { sFull = 0, sEmpty = 3, sSplit = 6, sP = 8, sGates = 10, sGFree = 12, sEnd = 14,
                  kStBars = 15 };

template <int NK, int TERMS>
struct StSmem {
  static constexpr uint32_t kWide = NK / 64 * kTile, kStage = kWide + kTile;
  static constexpr uint32_t oSplit = kStStages * kStage, oGates = oSplit + 2 * TERMS * kTile,
                            oBar = oGates + 2 * sizeof(Gates), oSlot = oBar + 8 * kStBars + 4,
                            oAbort = oSlot + 4, bytes = oAbort + 8;
  static constexpr uint32_t launch = bytes + 1024;
};

template <int NK, bool REV, int TERMS>
__global__ void __launch_bounds__(kStThreads, 1)
    decay_states_tc(const DecayArgs a, const DecaySplit sp, const __grid_constant__ CUtensorMap tx,
                    const __grid_constant__ CUtensorMap ty) {
  using L = StSmem<NK, TERMS>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slices = a.nv / 64, slice = blockIdx.x % slices;
  const int seg = blockIdx.x / slices + (REV ? sp.slot_of(1) : 0);   // (no gradient before)
  const int bh = blockIdx.y, b = bh / a.H, h = bh % a.H, hk = h / (a.H / a.Hk);
  const int t0 = seg * sp.piece_len, t1 = min(a.T, t0 + sp.piece_len);
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
  if (warp == 9) tc::tmem_alloc(smem_u32(slot), 256);
  if (tid == 0) {
    for (uint32_t i = 0; i < kStBars; ++i)
      tc::mbar_init(bar(i), (i >= sSplit && i < sP) || (i >= sGFree && i < sEnd) ? 8 : 1);   // warps
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

  auto split = [&](int n, int half) {
    if (!warp_wait(bar2(sGates, n), par(n), abort_flag) ||
        !warp_wait(bar(sFull + n % kStStages), (n / kStStages) & 1, abort_flag))
      return false;
    const Gates& g = gates(n);
    const float f = REV ? g.head[row] : g.tail[row];
#pragma unroll 1
    for (int c = 4 * half; c < 4 * half + 4; c += 2)
      split_row<TERMS>(sb + (n % kStStages) * L::kStage + L::kWide,
                       sb + L::oSplit + (n & 1) * TERMS * kTile, kTile, row, c, f);
    tc::fence_proxy_async();
    warp_arrive(bar2(sSplit, n));
    return true;
  };
  if (warp < 4) {
    float S[64];
    read_row(S, nullptr, 1);
    float sum = 0.f;
    bool ok = split(0, 0);
    for (int n = 0; ok && n < cnt; ++n) {
      if (n + 1 < cnt) ok = split(n + 1, 0);
      if (ok) ok = warp_wait(bar2(sP, n), par(n), abort_flag);
      if (!ok) break;
      tc::fence_after_sync();
      const float all = gates(n).all, add = gates(n).sum;
      warp_arrive(bar2(sGFree, n));
      if (mine || NK == 128) add_state(S, all, tl + (n & 1) * 128);
      sum += add;
      tc::fence_before_sync();
    }
    if (ok) {
      if (mine) write_row(S, REV ? a.scale : 1.f, dst + static_cast<size_t>(row) * a.nv);
      if (tid == 0 && slice == 0)   // (a piece of both walks: the same value twice)
        sp.decay[static_cast<size_t>(bh) * sp.pieces + seg] = decay_code(sum);
    }
  } else if (warp < 8) {
    for (int n = 0; n < cnt; ++n) {
      if (n >= 2 && !warp_wait(bar2(sP, n), par(n - 2), abort_flag)) break;
      if (!split(n, 1)) break;
      warp_arrive(bar2(sGFree, n));
    }
  } else if (warp == 8) {
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
  } else if (warp == 9) {
    const uint32_t go = lane == 0;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t idP = tc::idesc_bf16(128, 128, 1, 1);
    constexpr uint32_t idT = tc::idesc_bf16(128, 64, 1, 1);
    for (int n = 0; n < cnt; ++n) {
      // (the state has read this accumulator, chunk n - 2's, before it made this V')
      if (!warp_wait(bar2(sSplit, n), par(n), abort_flag)) break;
      tc::fence_after_sync();
      const uint64_t dx = tc::smem_desc(sb + (n % kStStages) * L::kStage, kTile, 1024);
      const uint64_t dy = tc::smem_desc(sb + L::oSplit + (n & 1) * TERMS * kTile, kTile, 1024);
      const uint64_t dt = tc::smem_desc(sb + L::oSplit + ((n & 1) * TERMS + 2) * kTile, 16, 1024);
#pragma unroll 1
      for (int k0 = 0; k0 < kC; k0 += 16) {
        const uint64_t at = (k0 * 128) >> 4;
        mma_if(go, tm + (n & 1) * 128, dx + at, dy + at, idP, k0 > 0);
        if (TERMS == 3) mma_if(go, tm + (n & 1) * 128 + 64, dx + at, dt + at, idT, 1);
      }
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
      fill_gates<false>(gates(n), x);
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
  if (warp == 9) tc::tmem_dealloc(tmem, 256);
}

// ------------------------------------------------------------------ pairs

// The pairs' part of the gate's gradient: with M_ri = s D_ri (q_r . k_i)
// (dO_r . v_i) over the pairs i < r of a chunk, for every token t, blocks of 32,
//   from_t = sum of M_ti over earlier blocks,   to_t = sum of M_rt over later ones,
//   near_t = sum of M_ti - sum of M_rt within t's block.
// Both products come twice, as they are and transposed, so that row sums and
// column sums are each a sum along one lane's columns; everything is fp32, as the
// sums' differences need it. The blocks' factors come out of the sums:
// from_t = row[t] sum_i (A . dA)_ti col[i].
// Chunks are independent: a CTA takes every ctas-th, and a chunk's
// tiles are asked for as soon as the products of the last one are complete.
// Warps 0-3: rows; 4-7: columns; 8: products and loads; 9: gates. As part of the
// backward's launch it fills the last wave (4 x 4096 x 16 x 128: 343 us in all).

enum : uint32_t { pFull = 0, pDone = 1, pFree = 2, pGates = 4, pGFree = 6, pEnd = 8, kPairBars = 9 };

template <int NK, int NV>
struct PairSmem {
  static constexpr uint32_t kK = NK / 64 * kTile, kV = NV / 64 * kTile;
  static constexpr uint32_t oQ = 0, oK = kK, oV = 2 * kK, oO = oV + kV, oGates = oO + kV,
                            oBar = oGates + 2 * sizeof(PairGates), oSlot = oBar + 8 * kPairBars,
                            oAbort = oSlot + 4, bytes = oAbort + 4;
  static constexpr uint32_t launch = bytes + 1024;
};

template <int NK, int NV>
__device__ __forceinline__ void pairs_cta(const DecayArgs& a, const DecaySplit& sp,
                                          const CUtensorMap* tq, const CUtensorMap* tk,
                                          const CUtensorMap* tv, const CUtensorMap* to, int cta,
                                          int ctas) {
  using L = PairSmem<NK, NV>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int chunks = (a.T + kC - 1) / kC;
  const long long jobs = static_cast<long long>(a.B) * a.H * chunks;
  const int cnt = jobs > cta ? static_cast<int>((jobs - cta + ctas - 1) / ctas) : 0;
  // heads fastest: heads that share q and k, and rows of one batch, run together
  auto job = [&](int n, int& b, int& h, int& t) {
    const long long j = cta + static_cast<long long>(n) * ctas;
    h = static_cast<int>(j % a.H);
    const long long c = j / a.H;
    t = static_cast<int>(c % chunks) * kC;
    b = static_cast<int>(c / chunks);
  };
  auto bar = [&](uint32_t i) { return sb + L::oBar + 8 * i; };
  auto bar2 = [&](uint32_t i, int n) { return bar(i + (n & 1)); };
  auto par = [](int n) { return static_cast<uint32_t>(n >> 1) & 1u; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::oAbort);
  uint32_t* slot = reinterpret_cast<uint32_t*>(smem + L::oSlot);
  auto gates = [&](int n) -> PairGates& {
    return *reinterpret_cast<PairGates*>(smem + L::oGates + (n & 1) * sizeof(PairGates));
  };
  if (warp == 8) tc::tmem_alloc(smem_u32(slot), 512);
  if (tid == 0) {
    for (uint32_t i = 0; i < kPairBars; ++i)
      tc::mbar_init(bar(i), i == pFree || i == pGFree || i == pGFree + 1 ? 8 : 1);   // warps
    *abort_flag = 0;
    tc::fence_mbar_init();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *slot;
  const int quad = warp & 3, row = 32 * quad + lane;
  const uint32_t tl = tmem + (static_cast<uint32_t>(32 * quad) << 16);
  const size_t plane = static_cast<size_t>(a.B) * a.H * a.T;

  if (warp < 8) {
    // rows: A, dA in columns 0 and 128; columns: their transposes in 256 and 384
    const bool cols = warp >= 4;
    const uint32_t ta = tl + (cols ? 256 : 0);
    float* far_out = (cols ? sp.to : sp.from) + (sp.flows - 1) * plane;
    float* near_out = sp.near + (cols ? plane : 0);
    for (int n = 0; n < cnt; ++n) {
      int b, h, t;
      job(n, b, h, t);
      if (!warp_wait(bar2(pGates, n), par(n), abort_flag) ||
          !warp_wait(bar(pDone), n & 1, abort_flag))
        break;
      tc::fence_after_sync();
      const PairGates& g = gates(n);
      const float lr = g.loc[row], ll = g.low[row];
      const uint32_t mine = g.allow[row];
      float far_sum = 0.f, near_sum = 0.f;
#pragma unroll 1
      for (int cb = cols ? quad : 0; cb <= (cols ? 3 : quad); ++cb) {
        float x[32], y[32];
        tc::tmem_ld32(ta + 32 * cb, x);
        tc::tmem_ld32(ta + 128 + 32 * cb, y);
        if (cb == quad) {
          const float *f = g.loc + 32 * cb, *fl = g.low + 32 * cb;
          const uint32_t* m = g.allow + 32 * cb;
          float acc[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            // rows: i < r reaches r; columns: r > i is reached by i
            const bool use = cols ? i > lane && (m[i] >> lane & 1u)
                                  : i < lane && (mine >> i & 1u);
            const float e = (f[i] - lr) + (fl[i] - ll);
            const float d = exp2_fast(cols ? e : -e);
            acc[i & 1] += use ? x[i] * y[i] * d : 0.f;
          }
          near_sum = acc[0] + acc[1];
        } else {
          const float fr = cols ? g.col[col_at(cb) + row] : g.row[row];
          const float* f = cols ? g.row + 32 * cb : g.col + col_at(quad) + 32 * cb;
          F2 acc[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const ulonglong2 c = *reinterpret_cast<const ulonglong2*>(f + i);
            acc[0] = fma2(mul2(pack2(x[i], x[i + 1]), pack2(y[i], y[i + 1])), c.x, acc[0]);
            acc[1] = fma2(mul2(pack2(x[i + 2], x[i + 3]), pack2(y[i + 2], y[i + 3])), c.y, acc[1]);
          }
          float u, v;
          unpack2(add2(acc[0], acc[1]), u, v);
          far_sum = fmaf(fr, u + v, far_sum);
        }
      }
      tc::fence_before_sync();
      warp_arrive(bar(pFree));
      warp_arrive(bar2(pGFree, n));
      if (t + row < a.T) {
        const size_t to_at = (static_cast<size_t>(b) * a.H + h) * a.T + t + row;
        far_out[to_at] = a.scale * far_sum;
        near_out[to_at] = (cols ? -a.scale : a.scale) * near_sum;
      }
    }
  } else if (warp == 8) {
    const uint32_t go = lane == 0;
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    constexpr uint32_t id = tc::idesc_bf16(128, 128, 0, 0);
    auto kmaj = [](int k0) { return static_cast<uint64_t>((k0 >> 6) * kTile + (k0 & 63) * 2) >> 4; };
    const uint64_t dq = tc::smem_desc(sb + L::oQ, 16, 1024), dk = tc::smem_desc(sb + L::oK, 16, 1024),
                   dv = tc::smem_desc(sb + L::oV, 16, 1024), dO = tc::smem_desc(sb + L::oO, 16, 1024);
    auto load = [&](int n) {
      int b, h, t;
      job(n, b, h, t);
      const int hk = h / (a.H / a.Hk);
      tc::mbar_arrive_expect_tx(bar(pFull), 2 * (L::kK + L::kV));
#pragma unroll
      for (int blk = 0; blk < NK / 64; ++blk) {
        tc::tma_load_4d(sb + L::oQ + blk * kTile, tq, 64 * blk, hk, t, b, bar(pFull));
        tc::tma_load_4d(sb + L::oK + blk * kTile, tk, 64 * blk, hk, t, b, bar(pFull));
      }
#pragma unroll
      for (int blk = 0; blk < NV / 64; ++blk) {
        tc::tma_load_4d(sb + L::oV + blk * kTile, tv, 64 * blk, h, t, b, bar(pFull));
        tc::tma_load_4d(sb + L::oO + blk * kTile, to, 64 * blk, h, t, b, bar(pFull));
      }
    };
    int issued = 0;
    if (cnt > 0) {
      if (lane == 0) load(0);
      issued = 1;
    }
    for (int n = 0; n < cnt; ++n) {
      if (!warp_wait(bar(pFull), n & 1, abort_flag)) break;
      if (n >= 1 && !warp_wait(bar(pFree), (n - 1) & 1, abort_flag)) break;
      tc::fence_after_sync();
#pragma unroll
      for (int k0 = 0; k0 < NK; k0 += 16) {
        mma_if(go, tm, dq + kmaj(k0), dk + kmaj(k0), id, k0 > 0);
        mma_if(go, tm + 256, dk + kmaj(k0), dq + kmaj(k0), id, k0 > 0);
      }
#pragma unroll
      for (int k0 = 0; k0 < NV; k0 += 16) {
        mma_if(go, tm + 128, dO + kmaj(k0), dv + kmaj(k0), id, k0 > 0);
        mma_if(go, tm + 384, dv + kmaj(k0), dO + kmaj(k0), id, k0 > 0);
      }
      commit_if(go, bar(pDone));
      if (n + 1 < cnt) {
        if (!warp_wait(bar(pDone), n & 1, abort_flag)) break;
        if (lane == 0) load(n + 1);
        issued = n + 2;
        __syncwarp();
      }
    }
    commit_if(go, bar(pEnd));
    tc::mbar_wait(bar(pEnd), 0);
    if (issued > 0) tc::mbar_wait(bar(pFull), (issued - 1) & 1);   // no copy may outlive the CTA
  } else if (warp == 9) {
    float x[4], y[4];
    auto read = [&](float (&v)[4], int n) {
      int b, h, t;
      job(n, b, h, t);
      read_gates(v, a, static_cast<size_t>(b) * a.T + t, h, min(kC, a.T - t));
    };
    if (cnt > 0) read(x, 0);
    for (int n = 0; n < cnt; ++n) {
      if (n + 1 < cnt) read(y, n + 1);
      if (n >= 2 && !warp_wait(bar2(pGFree, n), par(n - 2), abort_flag)) break;
      fill_gates<false>(gates(n), x);
      warp_arrive(bar2(pGates, n));
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = y[j];
    }
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (*abort_flag)   // a bounded wait gave up: this CTA's sums read NaN
    for (int n = 0; n < cnt; ++n) {
      int b, h, t;
      job(n, b, h, t);
      for (int i = tid; i < kC; i += kThreads)
        if (t + i < a.T)
          sp.near[(static_cast<size_t>(b) * a.H + h) * a.T + t + i] = __int_as_float(0x7fffffff);
    }
  if (warp == 8) tc::tmem_dealloc(tmem, 512);
}

// The whole backward: blockIdx.z 0: dq, 1: dk, 2: dv, from 3 on the pairs. They do
// not depend on one another, so in one launch they fill each other's last wave (the
// pairs come last, in CTAs of about four chunks), and with few sequences they run
// side by side (2 x 777 x 4 heads: 118 us as launches of their own, 62 as one).
// 4 x 4096 x 16 x 128: 343 us. What a chunk of dq or dk waits for is the chain P -> state
// -> R in three terms -> O1 next to Z' for the next P: issue slots are 0.37 busy, the
// load/store pipe 0.44 on the busiest SM, the tensor pipe 0.29, DRAM 0.40; of 11 warp
// cycles an instruction 4.4 are waits for a barrier or a read, 1.7 instruction fetch (0.78
// of the fetches hit) and 1.2 fixed latencies.
struct Walks {
  Walk dq, dk, dv;
};

template <int NK, int NV>
__global__ void __launch_bounds__(kThreads, 1)
    decay_bwd_tc(const DecayArgs a, const DecaySplit sp, const Walks w,
                 const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                 const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                 const __grid_constant__ CUtensorMap tdq, const __grid_constant__ CUtensorMap tdk) {
  const int x = blockIdx.x, bh = blockIdx.y;
  if (blockIdx.z >= 3) {
    const int plane = gridDim.x * gridDim.y;
    pairs_cta<NK, NV>(a, sp, &tq, &tk, &tv, &to,
                      (blockIdx.z - 3) * plane + bh * gridDim.x + x, (gridDim.z - 3) * plane);
    return;
  }
  const int slices = (blockIdx.z == 2 ? NV : NK) / 64;
  if (x >= sp.segments * slices) return;   // the other width has more slices
  if (blockIdx.z == 0)
    walk_cta<NV, false, true>(a, sp, w.dq, &to, &tv, &tk, &tdq, x / slices, x % slices, bh);
  else if (blockIdx.z == 1)
    walk_cta<NV, true, true>(a, sp, w.dk, &tv, &to, &tq, &tdk, x / slices, x % slices, bh);
  else
    walk_cta<NK, true, false>(a, sp, w.dv, &tk, &tq, &to, nullptr, x / slices, x % slices, bh);
}

template <class Kern>
cudaError_t opt_in(Kern kern, uint32_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(bytes));
}

struct Rows {   // one of the call's bf16 tensors
  const void* p;
  int heads, width;
  long long stride;
};
bool map_of(CUtensorMap* m, const DecayArgs& a, const Rows& r) {
  return make_rows_tmap(m, r.p, a.B, a.T, r.heads, r.width, r.stride);
}

template <int W>
cudaError_t fwd(const DecayArgs& a, const DecaySplit& sp, const Walk& w, const Rows& q,
                const Rows& k, const Rows& v, cudaStream_t stream) {
  using L = WalkSmem<W, false>;
  static_assert(L::launch <= 232448, "shared memory budget of one CTA");
  CUtensorMap tq, tk, tv;
  if (!map_of(&tq, a, q) || !map_of(&tk, a, k) || !map_of(&tv, a, v)) return cudaErrorInvalidValue;
  const cudaError_t err = opt_in(decay_fwd_tc<W>, L::launch);
  if (err != cudaSuccess) return err;
  decay_fwd_tc<W><<<dim3(sp.segments * (w.nz / 64), a.B * a.H), kThreads, L::launch, stream>>>(
      a, sp, w, tq, tk, tv);
  return cudaGetLastError();
}

// The walk's first state: S (or D), as rows of key channels or transposed, from
// the segments' chain or the caller's. D comes from the chain, which has copied dhT to
// its last slot, whenever there is one: dhT may be dh0, which the dv walk writes while
// the dk walk of the same launch reads its start.
Walk from(const DecayArgs& a, const DecaySplit& sp, bool grad, bool transposed) {
  Walk w{};
  const size_t st = static_cast<size_t>(a.nk) * a.nv;
  w.chained = grad ? sp.D != nullptr : sp.segments > 1;
  w.start = w.chained ? (grad ? sp.D : sp.S) : (grad ? nullptr : a.h0);
  w.start_bh = w.chained ? sp.slots * st : st;
  w.row_step = transposed ? 1 : a.nv;
  w.col_step = transposed ? a.nv : 1;
  return w;
}

template <int NK, bool REV, int TERMS>
cudaError_t states(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  using L = StSmem<NK, TERMS>;
  static_assert(L::launch <= 232448, "shared memory budget of one CTA");
  const long long so = static_cast<long long>(a.H) * a.nv;
  CUtensorMap tx, ty;
  if (!make_rows_tmap(&tx, REV ? a.q : a.k, a.B, a.T, a.Hk, NK, REV ? a.sq : a.sk) ||
      !make_rows_tmap(&ty, REV ? a.dO : a.v, a.B, a.T, a.H, a.nv, REV ? so : a.sv))
    return cudaErrorInvalidValue;
  const cudaError_t err = opt_in(decay_states_tc<NK, REV, TERMS>, L::launch);
  if (err != cudaSuccess) return err;
  const int segs = REV ? sp.pieces - sp.slot_of(1) : sp.states(a.dhT != nullptr);
  decay_states_tc<NK, REV, TERMS><<<dim3(segs * (a.nv / 64), a.B * a.H), kStThreads, L::launch, stream>>>(
      a, sp, tx, ty);
  return cudaGetLastError();
}

template <int NK, int NV>
cudaError_t bwd(const DecayArgs& a, const DecaySplit& sp, const Walks& w, const Rows& q,
                const Rows& k, const Rows& v, const Rows& dO, cudaStream_t stream) {
  constexpr uint32_t la = WalkSmem<NV, true>::launch, lb = WalkSmem<NK, false>::launch,
                     lc = PairSmem<NK, NV>::launch, lab = la > lb ? la : lb,
                     bytes = lab > lc ? lab : lc;
  static_assert(bytes <= 232448, "shared memory budget of one CTA");
  CUtensorMap tq, tk, tv, to, tdq, tdk;
  // (the maps of shared heads' gradients are not used: those leave as `part`)
  if (!map_of(&tq, a, q) || !map_of(&tk, a, k) || !map_of(&tv, a, v) || !map_of(&to, a, dO) ||
      !map_of(&tdq, a, {a.dq, a.Hk, NK, static_cast<long long>(a.Hk) * NK}) || !map_of(&tdk, a, {a.dk, a.Hk, NK, static_cast<long long>(a.Hk) * NK}))
    return cudaErrorInvalidValue;
  const cudaError_t err = opt_in(decay_bwd_tc<NK, NV>, bytes);
  if (err != cudaSuccess) return err;
  const int slices = (NK > NV ? NK : NV) / 64;
  const long long ctas = static_cast<long long>(sp.segments) * slices * a.B * a.H;
  const long long jobs = static_cast<long long>(a.B) * a.H * ((a.T + kC - 1) / kC);
  const int planes = static_cast<int>(std::max(1LL, std::min(16LL, jobs / (4 * ctas))));
  decay_bwd_tc<NK, NV><<<dim3(sp.segments * slices, a.B * a.H, 3 + planes), kThreads, bytes, stream>>>(
      a, sp, w, tq, tk, tv, to, tdq, tdk);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_fwd_tc(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  Walk w = from(a, sp, false, false);
  w.out = a.o;
  w.end = a.hT;
  w.x_heads = w.y_heads = a.Hk;
  w.z_heads = a.H;
  w.nz = a.nv;
  const Rows q{a.q, a.Hk, a.nk, a.sq}, k{a.k, a.Hk, a.nk, a.sk}, v{a.v, a.H, a.nv, a.sv};
  return a.nk == 64 ? fwd<64>(a, sp, w, q, k, v, stream) : fwd<128>(a, sp, w, q, k, v, stream);
}

cudaError_t launch_decay_bwd_tc(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream) {
  const Rows q{a.q, a.Hk, a.nk, a.sq}, k{a.k, a.Hk, a.nk, a.sk}, v{a.v, a.H, a.nv, a.sv},
      dO{a.dO, a.H, a.nv, static_cast<long long>(a.H) * a.nv};
  Walks w;
  w.dq = from(a, sp, false, true);
  w.dk = from(a, sp, true, true);
  w.dq.out = a.dq;
  w.dq.part = sp.dq_part;
  w.dq.z = w.dk.partner = static_cast<const __nv_bfloat16*>(a.k);
  w.dq.z_stride = w.dk.partner_stride = a.sk;
  w.dk.z = w.dq.partner = static_cast<const __nv_bfloat16*>(a.q);
  w.dk.z_stride = w.dq.partner_stride = a.sq;
  w.dq.flow = sp.from;
  w.dk.out = a.dk;
  w.dk.part = sp.dk_part;
  w.dk.flow = sp.to;
  for (Walk* p : {&w.dq, &w.dk}) {   // dO, v, k and v, dO, q
    p->x_heads = p->y_heads = a.H;
    p->z_heads = a.Hk;
    p->nz = a.nk;
  }
  w.dv = from(a, sp, true, false);   // k, q, dO
  w.dv.out = a.dv;
  w.dv.end = a.dh0;
  w.dv.x_heads = w.dv.y_heads = a.Hk;
  w.dv.z_heads = a.H;
  w.dv.nz = a.nv;
  if (a.nk == 64)
    return a.nv == 64 ? bwd<64, 64>(a, sp, w, q, k, v, dO, stream)
                      : bwd<64, 128>(a, sp, w, q, k, v, dO, stream);
  return a.nv == 64 ? bwd<128, 64>(a, sp, w, q, k, v, dO, stream)
                    : bwd<128, 128>(a, sp, w, q, k, v, dO, stream);
}

cudaError_t launch_decay_states_tc(const DecayArgs& a, const DecaySplit& sp, bool reverse,
                                   cudaStream_t stream) {
  if ((reverse ? sp.pieces - sp.slot_of(1) : sp.states(a.dhT != nullptr)) < 1) return cudaSuccess;
  // two terms for the forward, three where the gate's gradient comes from them (above)
  if (reverse)
    return a.nk == 64 ? states<64, true, 3>(a, sp, stream) : states<128, true, 3>(a, sp, stream);
  if (sp.D)
    return a.nk == 64 ? states<64, false, 3>(a, sp, stream) : states<128, false, 3>(a, sp, stream);
  return a.nk == 64 ? states<64, false, 2>(a, sp, stream) : states<128, false, 2>(a, sp, stream);
}

}  // namespace gdr
