// The C ABI of the block operators (declared in include/gdr.h): the short causal
// convolution, the state space recurrence and the norms after and before a block.
// Argument checks and kernel dispatch; nothing here allocates device memory or
// synchronises.
#include <algorithm>
#include <cmath>

#include "api_util.h"
#include "block_norms.h"
#include "short_conv.h"
#include "state_space.h"

namespace {

using gdr::align256;
using gdr::aligned;
using gdr::apart;
using gdr::check_workspace;
using gdr::given16;
using gdr::status_of;
using gdr::stream_of;

constexpr int kSms = 152;
constexpr int kMaxTokens = 1 << 30;
constexpr int kMaxChannels = 1 << 20;

// Elements between tokens as given (0: dense): at least `least`, whole 16 bytes.
gdr_status check_stride(long long given, long long least, int dtype) {
  const long long unit = dtype == GDR_BF16 ? 8 : 4;
  if (given != 0 && (given < least || given % unit != 0)) return GDR_ERR_INVALID_ARG;
  return given >= (1LL << 31) ? GDR_ERR_UNSUPPORTED : GDR_OK;
}

gdr_status check_conv(const gdr_conv_shape* s, bool step) {
  if (!s || s->B < 1 || s->T < 1 || s->D < 1 || s->K < 1) return GDR_ERR_INVALID_ARG;
  if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
  if (step && s->T != 1) return GDR_ERR_INVALID_ARG;
  if (s->K < 2 || s->K > 4 || s->D % 8 != 0 || s->D > kMaxChannels || s->T > kMaxTokens)
    return GDR_ERR_UNSUPPORTED;
  if (!step && s->B > 65535) return GDR_ERR_UNSUPPORTED;
  return check_stride(s->x_stride, s->D, s->dtype);
}

gdr::ConvArgs conv_args(const gdr_conv_shape* s) {
  gdr::ConvArgs a{};
  a.B = s->B; a.T = s->T; a.D = s->D; a.K = s->K;
  a.silu = s->silu != 0;
  a.xs = s->x_stride ? s->x_stride : s->D;
  return a;
}

gdr_status check_space(const gdr_state_space_shape* s, bool step) {
  if (!s || s->B < 1 || s->T < 1 || s->D < 1 || s->G < 1 || s->N < 1) return GDR_ERR_INVALID_ARG;
  if (s->dtype != GDR_F32 && s->dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
  if (s->D % s->G != 0 || (step && s->T != 1)) return GDR_ERR_INVALID_ARG;
  if (s->N != 8 && s->N != 16 && s->N != 32 && s->N != 64) return GDR_ERR_UNSUPPORTED;
  if (s->D / s->G % 8 != 0 || s->D > kMaxChannels || s->T > kMaxTokens || (!step && s->B > 65535))
    return GDR_ERR_UNSUPPORTED;
  const long long bc = static_cast<long long>(s->G) * s->N;
  const long long given[5] = {s->x_stride, s->dt_stride, s->z_stride, s->b_stride, s->c_stride};
  const long long least[5] = {s->D, s->D, s->D, bc, bc};
  for (int i = 0; i < 5; ++i) {
    const gdr_status st = check_stride(given[i], least[i], s->dtype);
    if (st != GDR_OK) return st;
  }
  return GDR_OK;
}

gdr::SpaceArgs space_args(const gdr_state_space_shape* s) {
  gdr::SpaceArgs a{};
  a.B = s->B; a.T = s->T; a.D = s->D; a.G = s->G; a.N = s->N;
  a.softplus = s->softplus != 0;
  const long long bc = static_cast<long long>(s->G) * s->N;
  a.xs = s->x_stride ? s->x_stride : s->D;
  a.dts = s->dt_stride ? s->dt_stride : s->D;
  a.zs = s->z_stride ? s->z_stride : s->D;
  a.bs = s->b_stride ? s->b_stride : bc;
  a.cs = s->c_stride ? s->c_stride : bc;
  return a;
}

// Time of n CTAs of equal length, `most` of which an SM holds at once: one takes `first`, each
// further one beside it `next` more.
double waves(long long n, int most, double first, double next) {
  const long long full = n / (kSms * most), rest = (n % (kSms * most) + kSms - 1) / kSms;
  return full * (first + next * (most - 1)) + (rest ? first + next * (rest - 1) : 0.0);
}

// Segments of each sequence. A CTA walks one segment of a batch row's channels, so few
// sequences are cut until the CTAs fill the SMs.
// Forward: uncut, a CTA has half the channels, and needs no other launch; a cut costs a walk
// over all segments but the last for their end states (0.65 of the other walk's time), and the
// chain. Times of a token (us, bf16, 16 states): uncut 0.084 and 0.054 (a CTA alone on its SM; a
// second one beside it), cut 0.17 and 0.055, and a third of a tile for a CTA's start; 3% more
// where all CTAs start together and stage their tiles in step. The further launches take 5 us one
// behind the other, and 8 of the host's. (1 x 512 x 4096 channels x 16: 45 us uncut, 29 in 16
// segments; 4 x 4096 x 4096: 542 uncut, 473 in 8 or 32 segments, 539 in 7; 1 x 65536 x 2048:
// 4961 uncut, 1046 in 19 segments, 938 in 38, 912 in 114.)
// The backward walks forward for its kept states anyway; a segment costs a CTA's start, 0.7
// tiles (4 x 4096 x 2048 x 16: 906 us in 4 segments, 794 in 14, 770 in 19, 764 in 24).
// fp32 and the other numbers of states are cut by the same times, though an SM holds three fp32
// CTAs where four and five are counted, and one in the gradients of 16 states where two are: the
// cut is near the best one all the same (4 x 4096 x 2048, against the best of 8 to 10 others:
// fp32 299 us for 290, 8 states 180 for 180, 32 443 for 439, 64 902 for 899; gradients in fp32
// 1060 for 1057, 8 states 633 for 629, 32 1346 for 1329, 64 2621 for 2586; the worst measured, fp32
// of 1 x 16384 x 2048, 309 for 291).
void cut(const gdr_state_space_shape* s, bool backward, gdr::SpaceSplit* sp) {
  const int tile = backward ? gdr::kSpaceTile : 32;
  const int tiles = (s->T + tile - 1) / tile, each = s->D / s->G;
  auto blocks = [&](int channels) { return (each + channels - 1) / channels; };
  sp->blocks = blocks(backward ? gdr::space_bwd_channels(s->N, s->dtype == GDR_F32)
                               : gdr::space_channels(s->N, false));
  const long long rows = static_cast<long long>(s->B) * s->G, ctas = rows * sp->blocks;
  double best = 0.0;
  int per = tiles;
  for (int n = 1; n <= 128 && n <= tiles; ++n) {
    const int len = (tiles + n - 1) / n, segments = (tiles + len - 1) / len;
    double cost;
    if (backward)
      cost = waves(ctas * segments, 2, 0.7, 0.3) * (len + 0.7);
    else if (segments == 1)
      cost = waves(rows * blocks(gdr::space_channels(s->N, true)), 2, 0.084, 0.054) * s->T;
    else
      cost = (waves(ctas * segments, 4, 0.17, 0.055) +
              0.65 * waves(ctas * (segments - 1), 5, 0.17, 0.055)) * (len + 0.3) * tile *
                 (1.0 + 0.03 * std::min(1.0, 4.0 * kSms / (ctas * segments))) + 13.0;
    if (n == 1 || cost < best) {
      best = cost;
      per = len;
    }
  }
  sp->segments = (tiles + per - 1) / per;
  sp->seg_len = per * tile;
  sp->tiles = tiles;
}

// Lays the arrays out from `base` (null: sizes only); returns the bytes used.
size_t lay_out(const gdr_state_space_shape* s, bool backward, char* base, gdr::SpaceSplit* sp) {
  size_t at = 0;
  auto take = [&](auto** p, size_t n) {
    if (base) *p = reinterpret_cast<std::remove_reference_t<decltype(*p)>>(base + at);
    at += align256(n * 4);
  };
  const size_t state = static_cast<size_t>(s->D) * s->N, B = s->B, D = s->D;
  const size_t runs = B * sp->segments;
  if (sp->segments > 1) {
    take(&sp->h, runs * state);
    take(&sp->total, runs * D);
    take(&sp->cleared, runs);
  }
  if (!backward) return at;
  if (sp->segments > 1) take(&sp->e, runs * state);
  take(&sp->kept, B * sp->tiles * state);
  take(&sp->kept_sum, B * sp->tiles * D);
  take(&sp->kept_clear, B * sp->tiles);
  take(&sp->dA_part, runs * state);
  take(&sp->d_part, runs * 2 * D);
  take(&sp->bc_part, B * s->T * s->G * 2 * s->N * sp->blocks);
  return at;
}

gdr_status check_norms(long long rows, int D, int dtype, float eps) {
  if (rows < 0 || D < 1) return GDR_ERR_INVALID_ARG;
  if (dtype != GDR_F32 && dtype != GDR_BF16) return GDR_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f) return GDR_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 8192 || rows > (1LL << 31) - 1) return GDR_ERR_UNSUPPORTED;
  return GDR_OK;
}

}  // namespace

extern "C" {

gdr_status gdr_short_conv_fwd(const gdr_conv_shape* shape, const void* x, const float* weight,
                              const float* bias, const unsigned char* starts, const void* state,
                              void* y, void* state_out, gdr_stream_t stream) {
  const gdr_status st = check_conv(shape, false);
  if (st != GDR_OK) return st;
  if (!given16(x) || !given16(weight) || !aligned(bias, 16) || !aligned(state, 16) || !given16(y) ||
      !aligned(state_out, 16) || !apart({y, state_out}, {x, weight, bias, starts, state}))
    return GDR_ERR_INVALID_ARG;
  gdr::ConvArgs a = conv_args(shape);
  a.x = x; a.weight = weight; a.bias = bias; a.starts = starts; a.state = state;
  a.y = y; a.state_out = state_out;
  return status_of(gdr::launch_short_conv(a, shape->dtype == GDR_F32, stream_of(stream)));
}

gdr_status gdr_short_conv_bwd_workspace(const gdr_conv_shape* shape, size_t* bytes) {
  const gdr_status st = check_conv(shape, false);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  *bytes = gdr::short_conv_bwd_workspace_bytes(shape->B, shape->T, shape->D, shape->K,
                                               shape->dtype == GDR_F32);
  return GDR_OK;
}

gdr_status gdr_short_conv_bwd(const gdr_conv_shape* shape, const void* x, const float* weight,
                              const float* bias, const unsigned char* starts, const void* state,
                              const void* dy, const void* dstate_out, void* dx, float* dweight,
                              float* dbias, void* dstate, void* workspace, size_t ws_bytes,
                              gdr_stream_t stream) {
  gdr_status st = check_conv(shape, false);
  if (st != GDR_OK) return st;
  if (!given16(x) || !given16(weight) || !aligned(bias, 16) || !aligned(state, 16) ||
      !given16(dy) || !aligned(dstate_out, 16) || !given16(dx) || !given16(dweight) ||
      !aligned(dbias, 16) || !aligned(dstate, 16))
    return GDR_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, gdr::short_conv_bwd_workspace_bytes(
                                                shape->B, shape->T, shape->D, shape->K,
                                                shape->dtype == GDR_F32));
  if (st != GDR_OK) return st;
  if (!apart({dx, dweight, dbias, dstate}, {x, weight, bias, starts, state, dy, dstate_out}))
    return GDR_ERR_INVALID_ARG;
  gdr::ConvArgs a = conv_args(shape);
  a.x = x; a.weight = weight; a.bias = bias; a.starts = starts; a.state = state;
  a.dy = dy; a.dstate_out = dstate_out; a.dx = dx; a.dweight = dweight; a.dbias = dbias;
  a.dstate = dstate; a.partial = static_cast<float*>(workspace);
  return status_of(gdr::launch_short_conv_bwd(a, shape->dtype == GDR_F32, stream_of(stream)));
}

gdr_status gdr_short_conv_step(const gdr_conv_shape* shape, const void* x, const float* weight,
                               const float* bias, void* state, void* y, gdr_stream_t stream) {
  const gdr_status st = check_conv(shape, true);
  if (st != GDR_OK) return st;
  if (!given16(x) || !given16(weight) || !aligned(bias, 16) || !given16(state) || !given16(y) ||
      !apart({y, state}, {x, weight, bias}))
    return GDR_ERR_INVALID_ARG;
  gdr::ConvArgs a = conv_args(shape);
  a.x = x; a.weight = weight; a.bias = bias; a.state_out = state; a.y = y;
  return status_of(gdr::launch_short_conv_step(a, shape->dtype == GDR_F32, stream_of(stream)));
}

gdr_status gdr_state_space_fwd_workspace(const gdr_state_space_shape* shape, size_t* bytes) {
  const gdr_status st = check_space(shape, false);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  gdr::SpaceSplit sp;
  cut(shape, false, &sp);
  *bytes = lay_out(shape, false, nullptr, &sp);
  return GDR_OK;
}

gdr_status gdr_state_space_fwd(const gdr_state_space_shape* shape, const void* x, const void* dt,
                               const float* A, const void* Bm, const void* Cm, const float* skip,
                               const void* z, const float* dt_bias, const unsigned char* starts,
                               const float* h0, void* y, float* hT, void* workspace,
                               size_t ws_bytes, gdr_stream_t stream) {
  gdr_status st = check_space(shape, false);
  if (st != GDR_OK) return st;
  if (!given16(x) || !given16(dt) || !given16(A) || !given16(Bm) || !given16(Cm) ||
      !aligned(skip, 16) || !aligned(z, 16) || !aligned(dt_bias, 16) || !aligned(h0, 16) ||
      !given16(y) || !aligned(hT, 16))
    return GDR_ERR_INVALID_ARG;
  gdr::SpaceSplit sp;
  cut(shape, false, &sp);
  st = check_workspace(workspace, ws_bytes, lay_out(shape, false, nullptr, &sp));
  if (st != GDR_OK) return st;
  // (hT may be h0)
  if (!apart({y, hT}, {x, dt, A, Bm, Cm, skip, z, dt_bias, starts}) || !apart({y}, {h0}))
    return GDR_ERR_INVALID_ARG;
  lay_out(shape, false, static_cast<char*>(workspace), &sp);
  gdr::SpaceArgs a = space_args(shape);
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.dt_bias = dt_bias;
  a.starts = starts; a.h0 = h0; a.y = y; a.hT = hT;
  const bool f32 = shape->dtype == GDR_F32;
  cudaError_t err = cudaSuccess;
  if (sp.segments > 1) {
    err = gdr::launch_space_states(a, sp, f32, stream_of(stream));
    if (err == cudaSuccess) err = gdr::launch_space_chain(a, sp, false, stream_of(stream));
  }
  if (err == cudaSuccess) err = gdr::launch_space_walk(a, sp, f32, stream_of(stream));
  return status_of(err);
}

gdr_status gdr_state_space_bwd_workspace(const gdr_state_space_shape* shape, size_t* bytes) {
  const gdr_status st = check_space(shape, false);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  gdr::SpaceSplit sp;
  cut(shape, true, &sp);
  *bytes = lay_out(shape, true, nullptr, &sp);
  return GDR_OK;
}

gdr_status gdr_state_space_bwd(const gdr_state_space_shape* shape, const void* x, const void* dt,
                               const float* A, const void* Bm, const void* Cm, const float* skip,
                               const void* z, const float* dt_bias, const unsigned char* starts,
                               const float* h0, const void* dy, const float* dhT, void* dx,
                               void* ddt, float* dA, void* dBm, void* dCm, float* dskip, void* dz,
                               float* ddt_bias, float* dh0, void* workspace, size_t ws_bytes,
                               gdr_stream_t stream) {
  gdr_status st = check_space(shape, false);
  if (st != GDR_OK) return st;
  if (!given16(x) || !given16(dt) || !given16(A) || !given16(Bm) || !given16(Cm) ||
      !aligned(skip, 16) || !aligned(z, 16) || !aligned(dt_bias, 16) || !aligned(h0, 16) ||
      !given16(dy) || !aligned(dhT, 16) || !given16(dx) || !given16(ddt) || !given16(dA) ||
      !given16(dBm) || !given16(dCm) || !aligned(dh0, 16) || (skip && !given16(dskip)) ||
      (z && !given16(dz)) || (dt_bias && !given16(ddt_bias)))
    return GDR_ERR_INVALID_ARG;
  gdr::SpaceSplit sp;
  cut(shape, true, &sp);
  st = check_workspace(workspace, ws_bytes, lay_out(shape, true, nullptr, &sp));
  if (st != GDR_OK) return st;
  // (dh0 may be dhT; what is not written may be anything)
  float* const gskip = skip ? dskip : nullptr;
  void* const gz = z ? dz : nullptr;
  float* const gbias = dt_bias ? ddt_bias : nullptr;
  if (!apart({dx, ddt, dA, dBm, dCm, gskip, gz, gbias, dh0},
             {x, dt, A, Bm, Cm, skip, z, dt_bias, starts, h0, dy}) ||
      !apart({dx, ddt, dA, dBm, dCm, gskip, gz, gbias}, {dhT}))
    return GDR_ERR_INVALID_ARG;
  lay_out(shape, true, static_cast<char*>(workspace), &sp);
  gdr::SpaceArgs a = space_args(shape);
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.dt_bias = dt_bias;
  a.starts = starts; a.h0 = h0; a.dy = dy; a.dhT = dhT;
  a.dx = dx; a.ddt = ddt; a.dA = dA; a.dBm = dBm; a.dCm = dCm; a.dskip = dskip; a.dz = dz;
  a.ddt_bias = ddt_bias; a.dh0 = dh0;
  const bool f32 = shape->dtype == GDR_F32;
  cudaError_t err = gdr::launch_space_bwd_states(a, sp, f32, stream_of(stream));
  if (err == cudaSuccess) err = gdr::launch_space_chain(a, sp, true, stream_of(stream));
  if (err == cudaSuccess) err = gdr::launch_space_bwd(a, sp, f32, stream_of(stream));
  return status_of(err);
}

gdr_status gdr_state_space_step(const gdr_state_space_shape* shape, const void* x, const void* dt,
                                const float* A, const void* Bm, const void* Cm, const float* skip,
                                const void* z, const float* dt_bias, float* state, void* y,
                                gdr_stream_t stream) {
  const gdr_status st = check_space(shape, true);
  if (st != GDR_OK) return st;
  if (!given16(x) || !given16(dt) || !given16(A) || !given16(Bm) || !given16(Cm) ||
      !aligned(skip, 16) || !aligned(z, 16) || !aligned(dt_bias, 16) || !given16(state) ||
      !given16(y) || !apart({y, state}, {x, dt, A, Bm, Cm, skip, z, dt_bias}))
    return GDR_ERR_INVALID_ARG;
  gdr::SpaceArgs a = space_args(shape);
  a.x = x; a.dt = dt; a.A = A; a.Bm = Bm; a.Cm = Cm; a.skip = skip; a.z = z; a.dt_bias = dt_bias;
  a.hT = state; a.y = y;
  return status_of(gdr::launch_space_step(a, shape->dtype == GDR_F32, stream_of(stream)));
}

gdr_status gdr_block_norms(long long rows, int D, gdr_dtype dtype, const void* x, const void* gate,
                           const void* residual, const float* post_weight, const float* scale,
                           const float* pre_weight, float eps, void* residual_out, void* y,
                           gdr_stream_t stream) {
  const gdr_status st = check_norms(rows, D, dtype, eps);
  if (st != GDR_OK) return st;
  if (rows == 0) return GDR_OK;
  if (!given16(x) || !aligned(gate, 16) || !given16(residual) || !given16(post_weight) ||
      !aligned(scale, 16) || !given16(pre_weight) || !given16(residual_out) || !given16(y) ||
      !apart({residual_out, y}, {post_weight, scale, pre_weight}))
    return GDR_ERR_INVALID_ARG;
  gdr::BlockNormsArgs a{x, gate, residual, post_weight, scale, pre_weight, residual_out, y, rows,
                        D, eps};
  return status_of(gdr::launch_block_norms(a, dtype == GDR_F32, stream_of(stream)));
}

gdr_status gdr_block_norms_bwd_workspace(long long rows, int D, size_t* bytes) {
  const gdr_status st = check_norms(rows, D, GDR_F32, 0.f);
  if (st != GDR_OK) return st;
  if (!bytes) return GDR_ERR_INVALID_ARG;
  *bytes = gdr::block_norms_bwd_workspace_bytes(rows, D);
  return GDR_OK;
}

gdr_status gdr_block_norms_bwd(long long rows, int D, gdr_dtype dtype, const void* dy,
                               const void* dres, const void* x, const void* gate, const void* sum,
                               const float* post_weight, const float* scale,
                               const float* pre_weight, float eps, void* dx, void* dgate,
                               void* dresidual, float* dpost, float* dscale, float* dpre,
                               void* workspace, size_t ws_bytes, gdr_stream_t stream) {
  gdr_status st = check_norms(rows, D, dtype, eps);
  if (st != GDR_OK) return st;
  if (!given16(post_weight) || !aligned(scale, 16) || !given16(pre_weight) || !given16(dpost) ||
      !given16(dpre) || (scale && !given16(dscale)))
    return GDR_ERR_INVALID_ARG;
  if (rows > 0 && (!given16(dy) || !aligned(dres, 16) || !given16(x) || !aligned(gate, 16) ||
                   !given16(sum) || !given16(dx) || !given16(dresidual) || dx == dresidual ||
                   (gate && (!given16(dgate) || dgate == dx || dgate == dresidual))))
    return GDR_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, gdr::block_norms_bwd_workspace_bytes(rows, D));
  if (st != GDR_OK) return st;
  // (rows may be written over rows of the inputs)
  float* const gscale = scale ? dscale : nullptr;
  if (!apart({dpost, gscale, dpre}, {post_weight, scale, pre_weight}) ||
      (rows > 0 && (!apart({dpost, gscale, dpre}, {dy, dres, x, gate, sum}) ||
                    !apart({dx, gate ? dgate : nullptr, dresidual, dpost, gscale, dpre},
                           {post_weight, scale, pre_weight}))))
    return GDR_ERR_INVALID_ARG;
  const cudaStream_t cs = stream_of(stream);
  if (rows == 0) {   // empty sums
    for (float* p : {dpost, scale ? dscale : dpre, dpre}) {
      const cudaError_t err = cudaMemsetAsync(p, 0, sizeof(float) * D, cs);
      if (err != cudaSuccess) return GDR_ERR_CUDA;
    }
    return GDR_OK;
  }
  gdr::BlockNormsBwdArgs a{dy, dres, x, gate, sum, post_weight, scale, pre_weight, dx, dgate,
                           dresidual, dpost, dscale, dpre, static_cast<float*>(workspace), rows, D,
                           eps};
  return status_of(gdr::launch_block_norms_bwd(a, dtype == GDR_F32, cs));
}

}  // extern "C"
