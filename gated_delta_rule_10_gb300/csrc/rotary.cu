// Rotary positions: channel pairs (x, y) of the first `rot` channels of a head
// turn by the token's angles,
//   (x, y) -> (x cos - y sin, y cos + x sin),
// the pair being channels (j, j + rot/2) or neighbours (2j, 2j + 1); the inverse
// turns back (sin negated), which is also the gradient. cos and sin are fp32
// tables over positions and j, made once by rotary_table_kernel in fp64.
//
// Bound by HBM: every element is read and written once. A thread takes 8 pairs
// (two 16-byte vectors of bf16) of kHeads heads of one token, q's and k's heads
// alike, so that one read of the 8 cosines and sines serves them all and kHeads
// pairs of loads are in flight: 44 us, 0.93 of measured HBM bandwidth, for
// 4 x 4096 x (16 + 16) heads x 128 (one head a thread, CTAs of 256: 58 us). A few
// tokens take as long as their launch.
#include "rotary.h"
#include "vec_io.cuh"

namespace gdr {
namespace {

constexpr int kHeads = 2;
constexpr int kThreads = 128;

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a, int units,
                                                          int groups, unsigned total) {
  const unsigned id = blockIdx.x * kThreads + threadIdx.x;
  if (id >= total) return;
  const int u = id % units;
  const unsigned rest = id / units;
  const int g = rest % groups;
  const long long tok = rest / groups;
  const int turned = a.rot / 16;
  // the unit's two vectors of 8 channels
  int c0, c1;
  if (u >= turned) {
    c0 = a.rot + 16 * (u - turned);
    c1 = c0 + 8;
  } else if (a.interleaved) {
    c0 = 16 * u;
    c1 = c0 + 8;
  } else {
    c0 = 8 * u;
    c1 = a.rot / 2 + 8 * u;
  }
  Raw8<T> raw[kHeads][2];
  const T* src[kHeads];
  T* dst[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    const int h = g + i * groups;
    const bool is_q = h < a.H;
    const int hk = h - a.H;
    src[i] = is_q ? static_cast<const T*>(a.q) + tok * a.sq + static_cast<long long>(h) * a.d
                  : static_cast<const T*>(a.k) + tok * a.sk + static_cast<long long>(hk) * a.d;
    dst[i] = is_q ? static_cast<T*>(a.q_out) + tok * a.sqo + static_cast<long long>(h) * a.d
                  : static_cast<T*>(a.k_out) + tok * a.sko + static_cast<long long>(hk) * a.d;
    if (h < a.H + a.Hk) {
      raw[i][0].load(src[i] + c0);
      raw[i][1].load(src[i] + c1);
    }
  }
  float x[2][8], cs[8], sn[8];
  if (u < turned) {
    const int p = a.pos ? __ldg(a.pos + tok) : a.start + static_cast<int>(tok % a.T);
    if (p >= 0 && p < a.table_len) {
      load8(a.cos_t + static_cast<long long>(p) * (a.rot / 2) + 8 * u, cs);
      load8(a.sin_t + static_cast<long long>(p) * (a.rot / 2) + 8 * u, sn);
    } else {   // no such row of the table: the result says so
#pragma unroll
      for (int j = 0; j < 8; ++j) cs[j] = sn[j] = __int_as_float(0x7fffffff);
    }
    if (a.inverse) {
#pragma unroll
      for (int j = 0; j < 8; ++j) sn[j] = -sn[j];
    }
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (g + i * groups >= a.H + a.Hk) continue;
    raw[i][0].get(x[0]);
    raw[i][1].get(x[1]);
    if (u < turned) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float& p0 = a.interleaved ? x[j >> 2][2 * (j & 3)] : x[0][j];
        float& p1 = a.interleaved ? x[j >> 2][2 * (j & 3) + 1] : x[1][j];
        const float e = p0, f = p1;
        p0 = e * cs[j] - f * sn[j];
        p1 = f * cs[j] + e * sn[j];
      }
    }
    store8(dst[i] + c0, x[0]);
    store8(dst[i] + c1, x[1]);
  }
}

// cos and sin of position p times the j-th frequency, in fp64 and rounded once.
// kind 0: base^(-2j/rot). 1: positions divided by `factor`. 2: the base raised so
// that the lowest frequency is divided by `factor`. 3 (the by-parts interpolation of
// "YaRN: Efficient Context Window Extension of Large Language Models", Peng et al.):
// frequencies that turn at least `fast` times over `original` positions are kept,
// those below `slow` are divided by `factor`, with a linear ramp in j between; cos and
// sin times `magnitude`. The ramp may end past the last frequency (half - 1): where even
// that one turns more than `slow` times, none is divided in full.
__global__ void __launch_bounds__(kThreads) rotary_table_kernel(const RotaryTableArgs a) {
  const long long id = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  const int half = a.rot / 2;
  if (id >= static_cast<long long>(a.len) * half) return;
  const int j = static_cast<int>(id % half);
  const double p = static_cast<double>(id / half), n = a.rot;
  double base = a.base;
  if (a.kind == 2 && a.rot > 2) base *= pow(a.factor, n / (n - 2.0));
  double f = pow(base, -2.0 * j / n);
  if (a.kind == 1) f /= a.factor;
  if (a.kind == 3) {
    const double two_pi = 6.283185307179586476925;
    // j at which a frequency turns r times over `original` positions
    auto at = [&](double r) {
      return n * log(a.original / (r * two_pi)) / (2.0 * log(a.base));
    };
    double lo = floor(at(a.fast)), hi = ceil(at(a.slow));
    lo = lo < 0.0 ? 0.0 : lo;
    hi = hi > n - 1.0 ? n - 1.0 : hi;
    double r = (j - lo) / (hi > lo ? hi - lo : 1e-3);
    r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
    f = f * (1.0 - r) + f / a.factor * r;
  }
  double s, c;
  sincos(p * f, &s, &c);
  a.cos_t[id] = static_cast<float>(c * a.magnitude);
  a.sin_t[id] = static_cast<float>(s * a.magnitude);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, bool f32, cudaStream_t stream) {
  const int units = (a.copy_tail ? a.d : a.rot) / 16;
  const int groups = (a.H + a.Hk + kHeads - 1) / kHeads;
  const long long total = a.tokens * units * groups;
  if (total > 2147483647LL) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>((total + kThreads - 1) / kThreads);
  if (f32)
    rotary_kernel<float><<<grid, kThreads, 0, stream>>>(a, units, groups,
                                                        static_cast<unsigned>(total));
  else
    rotary_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(a, units, groups,
                                                                static_cast<unsigned>(total));
  return cudaGetLastError();
}

cudaError_t launch_rotary_table(const RotaryTableArgs& a, cudaStream_t stream) {
  const long long n = static_cast<long long>(a.len) * (a.rot / 2);
  rotary_table_kernel<<<static_cast<unsigned>((n + kThreads - 1) / kThreads), kThreads, 0,
                        stream>>>(a);
  return cudaGetLastError();
}

}  // namespace gdr
