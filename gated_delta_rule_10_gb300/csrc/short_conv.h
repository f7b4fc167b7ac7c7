// Launch interface of the short causal convolution (short_conv.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr {

// Pointers as documented in include/gdr.h; xs is x's elements between tokens.
struct ConvArgs {
  const void *x, *state, *dy, *dstate_out;
  const float *weight, *bias;
  const unsigned char* starts;
  void *y, *state_out, *dx, *dstate;
  float *dweight, *dbias, *partial;
  int B, T, D, K;
  bool silu;
  long long xs;
};
size_t short_conv_bwd_workspace_bytes(int B, int T, int D, int K, bool f32);
cudaError_t launch_short_conv(const ConvArgs& a, bool f32, cudaStream_t stream);
cudaError_t launch_short_conv_bwd(const ConvArgs& a, bool f32, cudaStream_t stream);
cudaError_t launch_short_conv_step(const ConvArgs& a, bool f32, cudaStream_t stream);

}  // namespace gdr
