// Root-mean-square norm with the residual's addition, and its gradients.
//
//   r = round(x + res)            (stored in the inputs' type: the new residual)
//   y = r rsqrt(mean_c r_c^2 + eps) w
// y in the inputs' type, or in 8 bits (e4m3) with one fp32 scale for each 128
// columns: scale = max |y| / 448, at least 2^-126 (1 for a block of zeros), y8 =
// round(y (1 / scale)).
// For a gradient dy of y and dres of r (both may reach r), with inv = rsqrt(...):
//   dx = inv (w dy - r inv^2 mean_c(w dy r)) + dres,   dw = sum_rows dy r inv.
//
// Streams bound by HBM: every row is read once and stays in registers between
// its sums and the output. A row is spread over TPR threads (a warp up to a CTA of
// 512), at most kVec vectors of 8 columns per thread. The CTAs are persistent and
// walk the rows; the next row's vectors are requested before the current row's
// sums are taken, so that loads are in flight through the barriers and the stores
// (without: 334 us; with: 295 us, for 65536 x 4096 to 8 bits; 288 us, 0.97 of measured
// HBM, since a block's factor is all that its values take, with no division of theirs).
// The weight stays in registers over all rows.
#include <cuda_fp8.h>

#include <type_traits>

#include "add_rmsnorm.h"
#include "vec_io.cuh"

namespace gdr {
namespace {

constexpr int kVec = 2;          // 8-column vectors per thread, at most
constexpr float kE4m3Max = 448.f;
constexpr float kTiny = kE4m3Max * 1.17549435e-38f;   // 448 * 2^-126

template <typename T>
__device__ __forceinline__ float rounded(float x) {
  return static_cast<float>(static_cast<T>(x));
}

// Sums of two values over the TPR threads of a row (TPR a power of two from 32 to
// the CTA); `red` has a slot per warp and parity, so one barrier is enough.
template <int TPR>
__device__ __forceinline__ void row_sum(float& x, float& y, float2 (*red)[16], int parity) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, off);
    y += __shfl_xor_sync(0xffffffffu, y, off);
  }
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5, first = warp & ~(TPR / 32 - 1);
    if ((threadIdx.x & 31) == 0) red[parity][warp] = make_float2(x, y);
    __syncthreads();
    x = y = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      const float2 v = red[parity][first + i];
      x += v.x;
      y += v.y;
    }
  }
}

// A CTA has one row where a row takes 64 threads or more, so that rows do not wait
// for one another at the barrier.
template <int TPR>
constexpr int threads() { return TPR > 32 ? TPR : 256; }

template <typename T, int TPR, int VEC, bool FP8>
__global__ void __launch_bounds__(threads<TPR>(), sizeof(T) == 2 ? 768 / threads<TPR>() : 1)
    add_rmsnorm_kernel(const AddNormArgs a) {
  constexpr int kRows = threads<TPR>() / TPR;
  __shared__ float2 red[2][16];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nv = a.D / 8;          // vectors per row
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.res);
  float w[VEC][8];
  Raw8<T> rx[VEC], rr[VEC];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      if (row < a.rows && c < nv) {
        rx[i].load(x + row * a.D + 8 * c);
        rr[i].load(res + row * a.D + 8 * c);
      } else {
        rx[i].zero();
        rr[i].zero();
      }
    }
  };
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  long long r0 = static_cast<long long>(blockIdx.x) * kRows;
  fetch(r0 + sub);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = 0.f;
    if (c < nv) load8(a.weight + 8 * c, w[i]);
  }
  for (int parity = 0; r0 < a.rows; r0 += step, parity ^= 1) {
    const long long row = r0 + sub;
    const bool live = row < a.rows;
    float v[VEC][8];
    float ss = 0.f, none = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      float y[8];
      rx[i].get(v[i]);
      rr[i].get(y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] = rounded<T>(v[i][j] + y[j]);
        ss = fmaf(v[i][j], v[i][j], ss);
      }
      if (live && c < nv) store8(static_cast<T*>(a.res_out) + row * a.D + 8 * c, v[i]);
    }
    fetch(row + step);
    row_sum<TPR>(ss, none, red, parity);
    const float inv = rsqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      const bool in = live && c < nv;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * w[i][j];
      if (!FP8) {
        if (in) store8(static_cast<T*>(a.y) + row * a.D + 8 * c, v[i]);
      } else {
        // 128 columns are 16 neighbouring lanes; the largest magnitude is taken
        // as a NaN if one of them is
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          m = fmaxf(m, fabsf(v[i][j]));
          bad |= v[i][j] != v[i][j];
        }
        if (bad) m = __int_as_float(0x7fffffff);
#pragma unroll
        for (int off = 8; off > 0; off >>= 1) {
          const float o = __shfl_xor_sync(0xffffffffu, m, off);
          m = (o != o || o > m) ? o : m;
        }
        // y * (448 / max) is y / scale to one rounding. A subnormal scale would lose its
        // digits, or be zero (0 / 0): it stays at the smallest normal number
        const float scale = m == 0.f ? 1.f : m < kTiny ? kTiny / kE4m3Max : m / kE4m3Max;
        const float f = m < kTiny ? kE4m3Max / kTiny : kE4m3Max / m;
        if (in) {
          uint32_t p[2];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] *= f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[i][4 * j], v[i][4 * j + 1]),
                                                         __NV_SATFINITE, __NV_E4M3);
            const uint32_t hi = __nv_cvt_float2_to_fp8x2(
                make_float2(v[i][4 * j + 2], v[i][4 * j + 3]), __NV_SATFINITE, __NV_E4M3);
            p[j] = lo | (hi << 16);
          }
          __stcs(reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.y) + row * a.D + 8 * c),
                 make_uint2(p[0], p[1]));
          if ((c & 15) == 0) a.scales[row * ((a.D + 127) / 128) + c / 16] = scale;
        }
      }
    }
  }
}

// dx, and the weight's gradient of this CTA's rows as one row of `partial`. Each
// thread keeps its columns' sums in registers over all its rows; the CTA's row
// groups add theirs through shared memory at the end, in a fixed order. 512 threads of
// 128 registers an SM, which the grid counts on: with the ~150 that the compiler took by
// itself a quarter of the CTAs ran as a second wave (59 -> 51 us, 0.78 of measured HBM,
// for 16384 x 2048 bf16; ~5 of them are the second launch, which adds up the CTAs' rows).
template <typename T, int TPR, int VEC>
__global__ void __launch_bounds__(threads<TPR>(), 512 / threads<TPR>())
    add_rmsnorm_bwd_kernel(const AddNormBwdArgs a) {
  constexpr int kThreads = threads<TPR>(), kRows = kThreads / TPR;
  __shared__ float2 red[2][16];
  __shared__ float sums[kRows > 1 ? kThreads * 8 : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nv = a.D / 8;
  float w[VEC][8], dw[VEC][8];
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[i][j] = dw[i][j] = 0.f;
    if (c < nv) load8(a.weight + 8 * c, w[i]);
  }
  // rows are requested two ahead (fp32: one, which is as many bytes)
  constexpr int kDepth = sizeof(T) == 2 ? 2 : 1;
  struct Row {
    Raw8<T> x[VEC], y[VEC], d[VEC];
  } buf[kDepth];
  auto fetch = [&](Row& f, long long row) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      f.d[i].zero();
      if (row < a.rows && c < nv) {
        f.x[i].load(static_cast<const T*>(a.sum) + row * a.D + 8 * c);
        f.y[i].load(static_cast<const T*>(a.dy) + row * a.D + 8 * c);
        if (a.dres) f.d[i].load(static_cast<const T*>(a.dres) + row * a.D + 8 * c);
      } else {
        f.x[i].zero();
        f.y[i].zero();
      }
    }
  };
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  const long long r0 = static_cast<long long>(blockIdx.x) * kRows;
#pragma unroll
  for (int k = 0; k < kDepth; ++k) fetch(buf[k], r0 + sub + k * step);
  // (the row is widened once for its sums and once more for its output: as floats in
  // between it would not leave 128 registers for four rows of 2048 columns in flight)
  auto work = [&](Row& f, long long row, int parity) {
    const bool live = row < a.rows;
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float x[8], dy[8];
      f.x[i].get(x);
      f.y[i].get(dy);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(x[j], x[j], ss);
        dot = fmaf(w[i][j] * dy[j], x[j], dot);
      }
    }
    row_sum<TPR>(ss, dot, red, parity);
    const float n = static_cast<float>(a.D);
    const float inv = rsqrtf(ss / n + a.eps);
    const float m = inv * inv * (dot / n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      if (!(live && c < nv)) continue;
      float x[8], dy[8], d[8];
      f.x[i].get(x);
      f.y[i].get(dy);
      f.d[i].get(d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[i][j] = fmaf(dy[j], x[j] * inv, dw[i][j]);
        d[j] += inv * (w[i][j] * dy[j] - x[j] * m);
      }
      store8(static_cast<T*>(a.dx) + row * a.D + 8 * c, d);
    }
    fetch(f, row + kDepth * step);
  };
  for (long long r = r0; r < a.rows; r += 2 * step) {
    work(buf[0], r + sub, 0);
    if (r + step < a.rows) work(buf[kDepth - 1], r + step + sub, 1);
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
    if constexpr (kRows > 1) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) sums[threadIdx.x * 8 + j] = dw[i][j];
      __syncthreads();
      if (sub == 0)
        for (int r = 1; r < kRows; ++r)
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[i][j] += sums[(r * TPR + lane) * 8 + j];
    }
    if (sub == 0 && c < nv) {
      float* p = a.partial + static_cast<size_t>(blockIdx.x) * a.D + 8 * c;
      reinterpret_cast<float4*>(p)[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
    }
  }
}

// dw: column sums of the partial rows, in a fixed order. A CTA takes 32 columns,
// its 32 warps every 32nd row.
__global__ void __launch_bounds__(1024) weight_grad_kernel(const float* partial, float* dw, int D,
                                                           int n) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < D)
#pragma unroll 4
    for (int r = warp; r < n; r += 32) x += partial[static_cast<size_t>(r) * D + c];
  s[warp][lane] = x;
  __syncthreads();
  x = s[lane][warp];   // column `warp` of the block
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  if (lane == 0 && blockIdx.x * 32 + warp < D) dw[blockIdx.x * 32 + warp] = x;
}

// Threads per row and vectors per thread for a row of D columns.
template <class F>
cudaError_t by_width(int D, F f) {
  const int nv = D / 8;
  using std::integral_constant;
  if (nv <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (nv <= 64) return f(integral_constant<int, 32>{}, integral_constant<int, kVec>{});
  if (nv <= 128) return f(integral_constant<int, 64>{}, integral_constant<int, kVec>{});
  if (nv <= 256) return f(integral_constant<int, 128>{}, integral_constant<int, kVec>{});
  if (nv <= 512) return f(integral_constant<int, 256>{}, integral_constant<int, kVec>{});
  return f(integral_constant<int, 512>{}, integral_constant<int, kVec>{});
}

int ctas(long long rows, int per_cta, int most) {
  const long long want = (rows + per_cta - 1) / per_cta;
  return static_cast<int>(want < most ? want : most);
}

// CTAs of a kernel that all SMs hold at once, asked for once per device.
template <auto Kern>
int resident(int threads) {
  constexpr int kMaxDevices = 64;
  static int held[kMaxDevices] = {};
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return 1;
  if (held[dev] == 0 &&
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kern, threads, 0) == cudaSuccess)
    held[dev] = sms * per;
  return held[dev] > 0 ? held[dev] : 1;
}

template <typename T, int TPR, int VEC, bool FP8>
cudaError_t fwd_as(const AddNormArgs& a, cudaStream_t stream) {
  constexpr int kThreads = threads<TPR>(), kRows = kThreads / TPR;
  const int grid = ctas(a.rows, kRows, resident<add_rmsnorm_kernel<T, TPR, VEC, FP8>>(kThreads));
  add_rmsnorm_kernel<T, TPR, VEC, FP8><<<grid, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t fwd(const AddNormArgs& a, cudaStream_t stream) {
  return by_width(a.D, [&](auto tpr, auto vec) {
    return a.scales ? fwd_as<T, tpr, vec, true>(a, stream) : fwd_as<T, tpr, vec, false>(a, stream);
  });
}

template <typename T>
cudaError_t bwd(const AddNormBwdArgs& a, cudaStream_t stream) {
  return by_width(a.D, [&](auto tpr, auto vec) {
    constexpr int kThreads = threads<tpr>(), kRows = kThreads / tpr;
    const int grid = ctas(a.rows, kRows, kNormBwdCtas * 256 / kThreads);
    add_rmsnorm_bwd_kernel<T, tpr, vec><<<grid, kThreads, 0, stream>>>(a);
    weight_grad_kernel<<<(a.D + 31) / 32, 1024, 0, stream>>>(a.partial, a.dw, a.D, grid);
    return cudaGetLastError();
  });
}

}  // namespace

size_t add_rmsnorm_bwd_workspace_bytes(long long rows, int D) {
  size_t bytes = 0;
  by_width(D, [&](auto tpr, auto) {
    constexpr int kThreads = threads<tpr>(), kRows = kThreads / tpr;
    bytes = static_cast<size_t>(ctas(rows, kRows, kNormBwdCtas * 256 / kThreads)) * D *
            sizeof(float);
    return cudaSuccess;
  });
  return bytes;
}

cudaError_t launch_add_rmsnorm(const AddNormArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? fwd<float>(a, stream) : fwd<__nv_bfloat16>(a, stream);
}
cudaError_t launch_add_rmsnorm_bwd(const AddNormBwdArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? bwd<float>(a, stream) : bwd<__nv_bfloat16>(a, stream);
}

}  // namespace gdr
