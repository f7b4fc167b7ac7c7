// Launch interface of the norms after and before a block (block_norms.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr {

// Pointers as documented in include/gdr.h.
struct BlockNormsArgs {
  const void *x, *gate, *residual;
  const float *post, *scale, *pre;
  void *residual_out, *y;
  long long rows;
  int D;
  float eps;
};
struct BlockNormsBwdArgs {
  const void *dy, *dres, *x, *gate, *sum;
  const float *post, *scale, *pre;
  void *dx, *dgate, *dresidual;
  float *dpost, *dscale, *dpre, *partial;
  long long rows;
  int D;
  float eps;
};
size_t block_norms_bwd_workspace_bytes(long long rows, int D);
cudaError_t launch_block_norms(const BlockNormsArgs& a, bool f32, cudaStream_t stream);
cudaError_t launch_block_norms_bwd(const BlockNormsBwdArgs& a, bool f32, cudaStream_t stream);

}  // namespace gdr
