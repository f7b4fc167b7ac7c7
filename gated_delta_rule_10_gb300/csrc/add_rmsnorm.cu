// Root-mean-square norm with the residual's addition, and its gradients.
//
//   r = round(x + res)            (stored in the inputs' type: the new residual)
//   y = r rsqrt(mean_c r_c^2 + eps) w
// y in the inputs' type, or in 8 bits (e4m3) with one fp32 scale for each 128
// columns: scale = max |y| / 448 (1 for a block of zeros), y8 = round(y / scale).
// For a gradient dy of y and dres of r (both may reach r), with inv = rsqrt(...):
//   dx = inv (w dy - r inv^2 mean_c(w dy r)) + dres,   dw = sum_rows dy r inv.
//
// Streams bound by HBM: every row is read once and stays in registers between
// the sum of squares and the output. A row is spread over TPR threads (a warp up
// to a CTA), 8 columns (one 16-byte vector of bf16) per thread and step, at most
// kVec steps, so that wide rows keep as many loads in flight as narrow ones.
#include <cuda_fp8.h>

#include "add_rmsnorm.h"
#include "vec_io.cuh"

namespace gdr {
namespace {

constexpr int kVec = 4;          // 8-column vectors per thread, at most
constexpr float kE4m3Max = 448.f;

template <typename T>
__device__ __forceinline__ float rounded(float x) {
  return static_cast<float>(static_cast<T>(x));
}

// Sum over the TPR threads of a row (TPR a power of two from 32 to the CTA);
// `red` has one slot per warp and is free again at the next barrier.
template <int TPR>
__device__ __forceinline__ float row_sum(float x, float* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5, first = warp & ~(TPR / 32 - 1);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[warp] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) x += red[first + i];
  }
  return x;
}

template <typename T, int TPR, int VEC, bool FP8>
__global__ void __launch_bounds__(256) add_rmsnorm_kernel(const AddNormArgs a) {
  constexpr int kRows = 256 / TPR;
  __shared__ float red[8];
  const int lane = threadIdx.x % TPR;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const bool live = row < a.rows;
  const int nv = a.D / 8;          // vectors per row
  const T* x = static_cast<const T*>(a.x) + row * a.D;
  const T* res = static_cast<const T*>(a.res) + row * a.D;
  T* out = static_cast<T*>(a.res_out) + row * a.D;
  float v[VEC][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (live && c < nv) {
      float y[8];
      load8(x + 8 * c, v[i]);
      load8(res + 8 * c, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = rounded<T>(v[i][j] + y[j]);
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
    if (live && c < nv) store8(out + 8 * c, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  const float inv = rsqrtf(row_sum<TPR>(ss, red) / static_cast<float>(a.D) + a.eps);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
    const bool in = live && c < nv;
    float w[8] = {};
    if (in) load8(a.weight + 8 * c, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * w[j];
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
      const float scale = m == 0.f ? 1.f : m / kE4m3Max;
      if (in) {
        uint32_t p[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t lo = __nv_cvt_float2_to_fp8x2(
              make_float2(v[i][4 * j] / scale, v[i][4 * j + 1] / scale), __NV_SATFINITE,
              __NV_E4M3);
          const uint32_t hi = __nv_cvt_float2_to_fp8x2(
              make_float2(v[i][4 * j + 2] / scale, v[i][4 * j + 3] / scale), __NV_SATFINITE,
              __NV_E4M3);
          p[j] = lo | (hi << 16);
        }
        *reinterpret_cast<uint2*>(static_cast<unsigned char*>(a.y) + row * a.D + 8 * c) =
            make_uint2(p[0], p[1]);
        if ((c & 15) == 0) a.scales[row * ((a.D + 127) / 128) + c / 16] = scale;
      }
    }
  }
}

// dx, and the weight's gradient of this CTA's rows into one row of `partial`.
// Each thread keeps its columns' sums in registers over all its rows.
template <typename T, int TPR, int VEC>
__global__ void __launch_bounds__(256) add_rmsnorm_bwd_kernel(const AddNormBwdArgs a) {
  constexpr int kRows = 256 / TPR;
  __shared__ float red[8];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nv = a.D / 8;
  float dw[VEC][8];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  for (long long r0 = static_cast<long long>(blockIdx.x) * kRows; r0 < a.rows; r0 += step) {
    const long long row = r0 + sub;
    const bool live = row < a.rows;
    float x[VEC][8], dy[VEC][8];
    float ss = 0.f, dot = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[i][j] = dy[i][j] = 0.f;
      if (live && c < nv) {
        load8(static_cast<const T*>(a.sum) + row * a.D + 8 * c, x[i]);
        load8(static_cast<const T*>(a.dy) + row * a.D + 8 * c, dy[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      float w[8] = {};
      if (c < nv) load8(a.weight + 8 * c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(x[i][j], x[i][j], ss);
        dot = fmaf(w[j] * dy[i][j], x[i][j], dot);
      }
    }
    ss = row_sum<TPR>(ss, red);
    dot = row_sum<TPR>(dot, red);
    const float n = static_cast<float>(a.D);
    const float inv = rsqrtf(ss / n + a.eps);
    const float f = inv * inv * (dot / n);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      if (!(live && c < nv)) continue;
      float w[8], y[8] = {};
      load8(a.weight + 8 * c, w);
      if (a.dres) load8(static_cast<const T*>(a.dres) + row * a.D + 8 * c, y);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[i][j] = fmaf(dy[i][j], x[i][j] * inv, dw[i][j]);
        y[j] += inv * (w[j] * dy[i][j] - x[i][j] * f);
      }
      store8(static_cast<T*>(a.dx) + row * a.D + 8 * c, y);
    }
  }
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
    if (c < nv)
      store8(a.partial + (static_cast<size_t>(blockIdx.x) * kRows + sub) * a.D + 8 * c, dw[i]);
  }
}

// dw: column sums of the partial rows, in a fixed order. A CTA takes 32 columns,
// its eight warps every eighth row.
__global__ void __launch_bounds__(256) weight_grad_kernel(const float* partial, float* dw, int D,
                                                          int n) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < D)
    for (int r = warp; r < n; r += 8) x += partial[static_cast<size_t>(r) * D + c];
  s[warp][lane] = x;
  __syncthreads();
  if (warp == 0 && c < D) {
#pragma unroll
    for (int i = 1; i < 8; ++i) x += s[i][lane];
    dw[c] = x;
  }
}

// Threads per row and vectors per thread for a row of D columns.
template <class F>
cudaError_t by_width(int D, F f) {
  const int nv = D / 8;
  if (nv <= 32) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 1>{});
  if (nv <= 64) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 2>{});
  if (nv <= 128) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  if (nv <= 256) return f(std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{});
  if (nv <= 512) return f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 256>{}, std::integral_constant<int, kVec>{});
}

template <typename T>
cudaError_t fwd(const AddNormArgs& a, cudaStream_t stream) {
  return by_width(a.D, [&](auto tpr, auto vec) {
    constexpr int kRows = 256 / tpr;
    const long long grid = (a.rows + kRows - 1) / kRows;
    if (grid > 2147483647LL) return cudaErrorInvalidValue;
    if (a.scales)
      add_rmsnorm_kernel<T, tpr, vec, true><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
    else
      add_rmsnorm_kernel<T, tpr, vec, false><<<static_cast<unsigned>(grid), 256, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

// Partial rows of dw: enough CTAs to fill the GPU, each with at least a few rows.
int bwd_ctas(long long rows, int per_cta) {
  const long long want = (rows + per_cta - 1) / per_cta;
  return static_cast<int>(want < kNormBwdCtas ? want : kNormBwdCtas);
}

template <typename T>
cudaError_t bwd(const AddNormBwdArgs& a, cudaStream_t stream) {
  return by_width(a.D, [&](auto tpr, auto vec) {
    constexpr int kRows = 256 / tpr;
    const int grid = bwd_ctas(a.rows, kRows);
    add_rmsnorm_bwd_kernel<T, tpr, vec><<<grid, 256, 0, stream>>>(a);
    weight_grad_kernel<<<(a.D + 31) / 32, 256, 0, stream>>>(a.partial, a.dw, a.D, grid * kRows);
    return cudaGetLastError();
  });
}

}  // namespace

size_t add_rmsnorm_bwd_workspace_bytes(long long rows, int D) {
  size_t bytes = 0;
  by_width(D, [&](auto tpr, auto) {
    constexpr int kRows = 256 / tpr;
    bytes = static_cast<size_t>(bwd_ctas(rows, kRows)) * kRows * D * sizeof(float);
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
