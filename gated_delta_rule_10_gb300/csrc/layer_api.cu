// The C ABI of the layer operators around the delta rule (declared in
// include/gdr.h): linear attention with a decay for each head, the residual RMS
// norm and the rotary positions. Argument checks and kernel dispatch; nothing
// here allocates device memory or synchronises.
#include <stdint.h>

#include <cmath>

#include "add_rmsnorm.h"
#include "decay.h"
#include "gdr.h"
#include "rotary.h"

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
bool given16(const void* p) { return p && aligned(p, 16); }
size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
gdr_status status_of(cudaError_t err) { return err == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }
cudaStream_t stream_of(gdr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

constexpr int kSms = 152;
constexpr int kMaxTokens = 1 << 30;

gdr_status check_decay(const gdr_decay_shape* s, bool step) {
  if (!s) return GDR_ERR_INVALID_ARG;
  if (s->B < 1 || s->T < 1 || s->H < 1 || s->Hk < 1 || s->dk < 1 || s->dv < 1)
    return GDR_ERR_INVALID_ARG;
  if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
  if (!std::isfinite(s->scale) || s->H % s->Hk != 0) return GDR_ERR_INVALID_ARG;
  if (step && s->T != 1) return GDR_ERR_INVALID_ARG;
  if ((s->dk != 64 && s->dk != 128) || (s->dv != 64 && s->dv != 128)) return GDR_ERR_UNSUPPORTED;
  const long long unit = s->dtype == GDR_BF16 ? 8 : 4;   // 16 bytes
  const long long least[3] = {static_cast<long long>(s->Hk) * s->dk,
                              static_cast<long long>(s->Hk) * s->dk,
                              static_cast<long long>(s->H) * s->dv};
  const long long given[3] = {s->q_stride, s->k_stride, s->v_stride};
  for (int i = 0; i < 3; ++i)
    if (given[i] != 0 && (given[i] < least[i] || given[i] % unit != 0)) return GDR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (given[i] >= (1LL << 31)) return GDR_ERR_UNSUPPORTED;
  if (s->T > kMaxTokens) return GDR_ERR_UNSUPPORTED;
  const long long bh = static_cast<long long>(s->B) * s->H;
  if (step ? bh > 2147483647LL : bh > 65535) return GDR_ERR_UNSUPPORTED;   // grid extents
  return GDR_OK;
}

gdr::DecayArgs decay_args(const gdr_decay_shape* s) {
  gdr::DecayArgs a{};
  a.B = s->B; a.T = s->T; a.H = s->H; a.Hk = s->Hk; a.nk = s->dk; a.nv = s->dv;
  a.sq = s->q_stride ? s->q_stride : static_cast<long long>(s->Hk) * s->dk;
  a.sk = s->k_stride ? s->k_stride : static_cast<long long>(s->Hk) * s->dk;
  a.sv = s->v_stride ? s->v_stride : static_cast<long long>(s->H) * s->dv;
  a.per_head = s->decay_per_head != 0;
  a.scale = s->scale;
  return a;
}

constexpr int kMaxBwdRun = 4096;    // tokens per segment of the backward, at most

// Segments of each sequence, and pieces of each segment. A CTA walks one segment of
// a (batch, head, 64 columns), so few sequences are cut until the CTAs fill the
// SMs; each cut costs a pass over k and v for the segments' own states, so no
// further than that (1 x 65536 x 32 heads: two segments). That pass has one segment
// less, and takes segments in pieces until it fills the SMs too (864 -> 726 us).
// Segments are whole, so SMs stay idle where 152 is no multiple of the CTAs, and nothing
// is cut past 152: a token of a head at 128 x 128 in bf16 takes 0.22 ns with 152 CTAs,
// 0.26 with 128 or 256, 0.37 with 80 (1 x 8192 x 40 heads) or 160 (1 x 8192 x 80).
// The backward also bounds a segment's tokens: what its gate gradient passes on
// from block to block rounds (gate_grad_kernel), and its blocks are kept on chip.
void cut(const gdr_decay_shape* s, bool backward, gdr::DecaySplit* sp) {
  const int chunk = s->dtype == GDR_BF16 ? 128 : 64;
  const int chunks = (s->T + chunk - 1) / chunk;
  const long long ctas = static_cast<long long>(s->B) * s->H *
                         (s->dtype == GDR_BF16 ? s->dv / 64 : backward ? 2 : 1);
  long long p = kSms / ctas;
  // chunks per segment or piece, at least: a chunk takes ~2 us on the tensor cores,
  // less than the launches that a cut adds, and ~10 us in fp32, more than those
  // (1 x 257 x 2 heads x 64 in fp32: 63 us uncut, 31 us in five segments)
  const int least = s->dtype == GDR_BF16 ? 4 : 1;
  if (p > chunks / least) p = chunks / least;
  if (backward && p < (s->T + kMaxBwdRun - 1) / kMaxBwdRun)
    p = (s->T + kMaxBwdRun - 1) / kMaxBwdRun;
  if (p < 1) p = 1;
  int per = static_cast<int>((chunks + p - 1) / p);
  sp->segments = (chunks + per - 1) / per;
  long long q = 1;
  if (sp->segments > 1) {
    const long long busy = ctas * (sp->segments - 1);
    q = kSms / busy;
    if (q > per / least) q = per / least;
    if (q < 1) q = 1;
  }
  const int piece = static_cast<int>((per + q - 1) / q);
  per = static_cast<int>(piece * q);       // whole pieces
  if (backward && per * chunk > kMaxBwdRun) {
    per = piece * (kMaxBwdRun / chunk / piece);
    if (per < 1) per = kMaxBwdRun / chunk;
  }
  sp->segments = (chunks + per - 1) / per;
  sp->parts_per = per / piece;
  sp->piece_len = piece * chunk;
  sp->seg_len = per * chunk;
  sp->pieces = sp->segments > 1 ? (chunks + piece - 1) / piece : 1;
  if (sp->segments == 1) {   // one piece, whose state only the backward needs
    sp->parts_per = 1;
    sp->piece_len = sp->seg_len;
  }
  sp->parts = s->dk * s->dv / 1024;
}

// Lays the arrays out from `base` (null: sizes only); returns the bytes used.
size_t lay_out(const gdr_decay_shape* s, bool backward, bool end_grad, char* base,
               gdr::DecaySplit* sp) {
  size_t at = 0;
  auto take = [&](float** p, size_t n) {
    if (base) *p = reinterpret_cast<float*>(base + at);
    at += align256(n * sizeof(float));
  };
  const size_t bh = static_cast<size_t>(s->B) * s->H, st = static_cast<size_t>(s->dk) * s->dv;
  const bool chain = sp->segments > 1 || (backward && end_grad);
  sp->slots = sp->pieces + (backward ? 1 : 0);
  if (chain) {
    take(&sp->S, bh * sp->slots * st);
    take(&sp->decay, bh * sp->pieces);
  }
  if (!backward) return at;
  if (chain) {
    take(&sp->D, bh * sp->slots * st);
    take(&sp->dots, bh * sp->slots * sp->parts);
  }
  const bool tc = s->dtype == GDR_BF16;
  sp->flows = tc ? s->dk / 64 + 1 : 2;   // the states' parts (by column slice), and the pairs
  sp->nears = tc ? 2 : 1;                // rows, columns
  sp->firsts = tc ? s->dk / 64 * (s->dv / 32) : 1;   // a warp of each column slice's
  take(&sp->first, bh * sp->firsts);
  take(&sp->from, sp->flows * bh * s->T);
  take(&sp->to, sp->flows * bh * s->T);
  take(&sp->near, sp->nears * bh * s->T);
  if (s->Hk != s->H) {
    take(&sp->dq_part, bh * s->T * s->dk);
    take(&sp->dk_part, bh * s->T * s->dk);
  }
  if (s->decay_per_head) take(&sp->dg_part, bh * sp->segments);
  return at;
}

gdr_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return GDR_OK;
  if (!ws || have < need) return GDR_ERR_WORKSPACE;
  return aligned(ws, 16) ? GDR_OK : GDR_ERR_INVALID_ARG;
}

gdr_status check_norm(long long rows, int D, int dtype, float eps) {
  if (rows < 0 || D < 1) return GDR_ERR_INVALID_ARG;
  if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return GDR_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > gdr::kNormMaxWidth || rows > (1LL << 31) - 1) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

gdr_status add_rmsnorm(long long rows, int D, int dtype, const void* x, const void* residual,
                       const float* weight, float eps, void* residual_out, void* y, float* scales,
                       bool fp8, gdr_stream_t stream) {
  const gdr_status st = check_norm(rows, D, dtype, eps);
  if (st != GDR_OK) return st;
  if (rows == 0) return GDR_OK;
  if (!given16(x) || !given16(residual) || !given16(weight) || !given16(residual_out) ||
      !given16(y) || (fp8 && (!scales || !aligned(scales, 4))))
    return GDR_ERR_INVALID_ARG;
  gdr::AddNormArgs a{x, residual, weight, residual_out, y, fp8 ? scales : nullptr, rows, D, eps};
  return status_of(gdr::launch_add_rmsnorm(a, dtype == GDR_F32, stream_of(stream)));
}

}  // namespace

extern "C" {

gdr_status gdr_decay_chunk_fwd_workspace(const gdr_decay_shape* shape, size_t* bytes) {
  const gdr_status st = check_decay(shape, false);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  gdr::DecaySplit sp;
  cut(shape, false, &sp);
  *bytes = lay_out(shape, false, false, nullptr, &sp);
  return GDR_OK;
}

gdr_status gdr_decay_chunk_fwd(const gdr_decay_shape* shape, const void* q, const void* k,
                               const void* v, const float* g, const float* h0, void* o, float* hT,
                               void* workspace, size_t ws_bytes, gdr_stream_t stream) {
  gdr_status st = check_decay(shape, false);
  if (st != GDR_OK) return st;
  if (!given16(q) || !given16(k) || !given16(v) || !given16(o) || !g || !aligned(g, 4) ||
      !aligned(h0, 16) || !aligned(hT, 16))
    return GDR_ERR_INVALID_ARG;
  gdr::DecaySplit sp;
  cut(shape, false, &sp);
  st = check_workspace(workspace, ws_bytes, lay_out(shape, false, false, nullptr, &sp));
  if (st != GDR_OK) return st;
  lay_out(shape, false, false, static_cast<char*>(workspace), &sp);
  gdr::DecayArgs a = decay_args(shape);
  a.q = q; a.k = k; a.v = v; a.g = g; a.h0 = h0; a.o = o; a.hT = hT;
  const bool f32 = shape->dtype == GDR_F32;
  const cudaStream_t cs = stream_of(stream);
  cudaError_t err = cudaSuccess;
  if (sp.segments > 1) {
    err = f32 ? gdr::launch_decay_states_f32(a, sp, false, cs)
              : gdr::launch_decay_states_tc(a, sp, false, cs);
    if (err == cudaSuccess) err = gdr::launch_decay_chain(a, sp, false, cs);
  }
  if (err == cudaSuccess)
    err = f32 ? gdr::launch_decay_fwd_f32(a, sp, cs) : gdr::launch_decay_fwd_tc(a, sp, cs);
  return status_of(err);
}

gdr_status gdr_decay_chunk_bwd_workspace(const gdr_decay_shape* shape, size_t* bytes) {
  const gdr_status st = check_decay(shape, false);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  gdr::DecaySplit sp;
  cut(shape, true, &sp);
  *bytes = lay_out(shape, true, true, nullptr, &sp);
  return GDR_OK;
}

gdr_status gdr_decay_chunk_bwd(const gdr_decay_shape* shape, const void* q, const void* k,
                               const void* v, const float* g, const float* h0, const void* dO,
                               const float* dhT, void* dq, void* dk, void* dv, float* dg,
                               float* dh0, void* workspace, size_t ws_bytes,
                               gdr_stream_t stream) {
  gdr_status st = check_decay(shape, false);
  if (st != GDR_OK) return st;
  if (!given16(q) || !given16(k) || !given16(v) || !given16(dO) || !given16(dq) || !given16(dk) ||
      !given16(dv) || !g || !aligned(g, 4) || !dg || !aligned(dg, 4) || !aligned(h0, 16) ||
      !aligned(dhT, 16) || !aligned(dh0, 16))
    return GDR_ERR_INVALID_ARG;
  gdr::DecaySplit sp;
  cut(shape, true, &sp);
  st = check_workspace(workspace, ws_bytes, lay_out(shape, true, true, nullptr, &sp));
  if (st != GDR_OK) return st;
  lay_out(shape, true, dhT != nullptr, static_cast<char*>(workspace), &sp);
  gdr::DecayArgs a = decay_args(shape);
  a.q = q; a.k = k; a.v = v; a.g = g; a.h0 = h0; a.dO = dO; a.dhT = dhT;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dh0 = dh0;
  const bool f32 = shape->dtype == GDR_F32;
  const cudaStream_t cs = stream_of(stream);
  cudaError_t err = cudaSuccess;
  if (sp.S) {
    for (int rev = 0; rev < 2 && err == cudaSuccess; ++rev)
      err = f32 ? gdr::launch_decay_states_f32(a, sp, rev, cs)
                : gdr::launch_decay_states_tc(a, sp, rev, cs);
    if (err == cudaSuccess) err = gdr::launch_decay_chain(a, sp, true, cs);
  }
  if (err == cudaSuccess)
    err = f32 ? gdr::launch_decay_bwd_f32(a, sp, cs) : gdr::launch_decay_bwd_tc(a, sp, cs);
  if (err == cudaSuccess) err = gdr::launch_decay_gate_grad(a, sp, f32, cs);
  return status_of(err);
}

gdr_status gdr_decay_step(const gdr_decay_shape* shape, const void* q, const void* k,
                          const void* v, const float* g, float* state, void* o,
                          gdr_stream_t stream) {
  const gdr_status st = check_decay(shape, true);
  if (st != GDR_OK) return st;
  if (!given16(q) || !given16(k) || !given16(v) || !given16(o) || !given16(state) || !g ||
      !aligned(g, 4))
    return GDR_ERR_INVALID_ARG;
  const gdr::DecayArgs d = decay_args(shape);
  gdr::DecayStepArgs a{q, k, v, g, state, o, shape->B, shape->H, shape->Hk, d.sq, d.sk, d.sv,
                       d.per_head, shape->scale};
  return status_of(gdr::launch_decay_step(a, shape->dk, shape->dv, shape->dtype == GDR_F32,
                                          stream_of(stream)));
}

gdr_status gdr_add_rmsnorm(long long rows, int D, gdr_dtype dtype, const void* x,
                           const void* residual, const float* weight, float eps,
                           void* residual_out, void* y, gdr_stream_t stream) {
  return add_rmsnorm(rows, D, dtype, x, residual, weight, eps, residual_out, y, nullptr, false,
                     stream);
}

gdr_status gdr_add_rmsnorm_fp8(long long rows, int D, gdr_dtype dtype, const void* x,
                               const void* residual, const float* weight, float eps,
                               void* residual_out, void* y, float* scales, gdr_stream_t stream) {
  return add_rmsnorm(rows, D, dtype, x, residual, weight, eps, residual_out, y, scales, true,
                     stream);
}

gdr_status gdr_add_rmsnorm_bwd_workspace(long long rows, int D, size_t* bytes) {
  const gdr_status st = check_norm(rows, D, GDR_F32, 0.f);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  *bytes = gdr::add_rmsnorm_bwd_workspace_bytes(rows, D);
  return GDR_OK;
}

gdr_status gdr_add_rmsnorm_bwd(long long rows, int D, gdr_dtype dtype, const void* dy,
                               const void* sum, const float* weight, float eps, const void* dres,
                               void* dx, float* dweight, void* workspace, size_t ws_bytes,
                               gdr_stream_t stream) {
  gdr_status st = check_norm(rows, D, dtype, eps);
  if (st != GDR_OK) return st;
  if (!given16(weight) || !given16(dweight)) return GDR_ERR_INVALID_ARG;
  if (rows > 0 && (!given16(dy) || !given16(sum) || !given16(dx) || !aligned(dres, 16)))
    return GDR_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, gdr::add_rmsnorm_bwd_workspace_bytes(rows, D));
  if (st != GDR_OK) return st;
  if (rows == 0)   // an empty sum
    return status_of(cudaMemsetAsync(dweight, 0, sizeof(float) * D, stream_of(stream)));
  gdr::AddNormBwdArgs a{dy, sum, dres, weight, dx, dweight, static_cast<float*>(workspace), rows,
                        D, eps};
  return status_of(gdr::launch_add_rmsnorm_bwd(a, dtype == GDR_F32, stream_of(stream)));
}

gdr_status gdr_rotary_table(int length, int rot, double base, const gdr_rotary_scaling* scaling,
                            float* cos_table, float* sin_table, gdr_stream_t stream) {
  if (length < 1 || rot < 16 || rot % 16 != 0 || !(base > 1.0) || !std::isfinite(base))
    return GDR_ERR_INVALID_ARG;
  if (!given16(cos_table) || !given16(sin_table)) return GDR_ERR_INVALID_ARG;
  gdr::RotaryTableArgs a{cos_table, sin_table, length, rot, 0, base, 1.0, 1.0, 1.0, 1.0, 1.0};
  if (scaling) {
    if (scaling->kind < GDR_ROPE_NONE || scaling->kind > GDR_ROPE_RAMP) return GDR_ERR_INVALID_ARG;
    if (scaling->kind != GDR_ROPE_NONE &&
        (!(scaling->factor >= 1.0) || !std::isfinite(scaling->factor)))
      return GDR_ERR_INVALID_ARG;
    a.kind = scaling->kind;
    if (a.kind != GDR_ROPE_NONE) a.factor = scaling->factor;
    if (a.kind == GDR_ROPE_RAMP) {
      if (scaling->original_length < 1 || !(scaling->fast > scaling->slow) ||
          !(scaling->slow > 0.0) || !std::isfinite(scaling->fast) ||
          !(scaling->magnitude > 0.0) || !std::isfinite(scaling->magnitude))
        return GDR_ERR_INVALID_ARG;
      a.original = scaling->original_length;
      a.fast = scaling->fast;
      a.slow = scaling->slow;
      a.magnitude = scaling->magnitude;
    }
  }
  return status_of(gdr::launch_rotary_table(a, stream_of(stream)));
}

gdr_status gdr_rotary(const gdr_rotary_shape* s, const void* q, const void* k,
                      const float* cos_table, const float* sin_table, const int* positions,
                      void* q_out, void* k_out, gdr_stream_t stream) {
  if (!s || s->B < 0 || s->T < 0 || s->H < 0 || s->Hk < 0 || s->H + static_cast<long long>(s->Hk) < 1)
    return GDR_ERR_INVALID_ARG;
  if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
  if (s->rot < 16 || s->rot % 16 != 0 || s->rot > s->d || s->table_length < 1)
    return GDR_ERR_INVALID_ARG;
  if (s->d % 16 != 0 || s->d > 65536 || s->H > 65536 || s->Hk > 65536) return GDR_ERR_UNSUPPORTED;
  const long long unit = s->dtype == GDR_BF16 ? 8 : 4;
  const long long wq = static_cast<long long>(s->H) * s->d, wk = static_cast<long long>(s->Hk) * s->d;
  const long long given[4] = {s->q_stride, s->k_stride, s->q_out_stride, s->k_out_stride};
  const long long least[4] = {wq, wk, wq, wk};
  for (int i = 0; i < 4; ++i)
    if (given[i] != 0 && (given[i] < least[i] || given[i] % unit != 0)) return GDR_ERR_INVALID_ARG;
  const long long tokens = static_cast<long long>(s->B) * s->T;
  if (tokens == 0) return GDR_OK;
  if ((s->H > 0 && (!given16(q) || !given16(q_out))) ||
      (s->Hk > 0 && (!given16(k) || !given16(k_out))))
    return GDR_ERR_INVALID_ARG;
  if (!given16(cos_table) || !given16(sin_table) || !aligned(positions, 4))
    return GDR_ERR_INVALID_ARG;
  // threads: one per token, 16 channels and 2 heads
  if (tokens > (1LL << 31) - 1 ||
      tokens * (s->d / 16) * ((s->H + static_cast<long long>(s->Hk) + 1) / 2) > (1LL << 31) - 257)
    return GDR_ERR_UNSUPPORTED;
  gdr::RotaryArgs a{};
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.cos_t = cos_table; a.sin_t = sin_table; a.pos = positions;
  a.tokens = tokens; a.T = s->T; a.H = s->H; a.Hk = s->Hk; a.d = s->d; a.rot = s->rot;
  a.start = s->start; a.table_len = s->table_length;
  a.sq = s->q_stride ? s->q_stride : wq;
  a.sk = s->k_stride ? s->k_stride : wk;
  a.sqo = s->q_out_stride ? s->q_out_stride : wq;
  a.sko = s->k_out_stride ? s->k_out_stride : wk;
  a.interleaved = s->interleaved != 0;
  a.inverse = s->inverse != 0;
  // in place, the channels past rot already hold their values
  a.copy_tail = (s->H > 0 && q != q_out) || (s->Hk > 0 && k != k_out);
  return status_of(gdr::launch_rotary(a, s->dtype == GDR_F32, stream_of(stream)));
}

}  // extern "C"
