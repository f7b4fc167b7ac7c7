// Column sums of a gradient's partial rows, in a fixed order: a CTA takes 32 columns, its
// 32 warps every 32nd row; `put(column, sum)` stores the result.
#pragma once

#include <cuda_runtime.h>

namespace gdr {

template <class Put>
__device__ __forceinline__ void column_sum(const float* partial, int rows, int columns, Put put) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < columns)
#pragma unroll 4
    for (int r = warp; r < rows; r += 32) x += partial[static_cast<size_t>(r) * columns + c];
  s[warp][lane] = x;
  __syncthreads();
  x = s[lane][warp];   // column `warp` of the block
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  if (lane == 0 && blockIdx.x * 32 + warp < columns) put(blockIdx.x * 32 + warp, x);
}

}  // namespace gdr
