// Column sums of a gradient's partial rows, in a fixed order: a CTA takes 32 columns, each of
// its WARPS warps every WARPS-th row; `put(column, sum)` stores the result. More warps wait
// less for few columns' rows, fewer let more CTAs run at once (the filter's gradient of 4 x 4096 x
// 4096, 36 rows of 20480 columns: 8 warps 2 us faster than 32; the norms', 304 of 4096: 2 slower).
#pragma once

#include <cuda_runtime.h>

namespace gdr {

template <int WARPS, class Put>
__device__ __forceinline__ void column_sum(const float* partial, int rows, int columns, Put put) {
  constexpr int kOwn = 32 / WARPS;      // columns that a warp finishes
  __shared__ float s[WARPS][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < columns)
#pragma unroll 8
    for (int r = warp; r < rows; r += WARPS) x += partial[static_cast<size_t>(r) * columns + c];
  s[warp][lane] = x;
  __syncthreads();
  const int own = warp * kOwn + lane / WARPS;
  x = s[lane % WARPS][own];
#pragma unroll
  for (int off = WARPS / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  if (lane % WARPS == 0 && blockIdx.x * 32 + own < columns) put(blockIdx.x * 32 + own, x);
}

}  // namespace gdr
