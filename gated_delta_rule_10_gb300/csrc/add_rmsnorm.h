// Launch interface of the residual RMS norm and its gradients (add_rmsnorm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr {

constexpr int kNormMaxWidth = 8192;   // columns of a row: what a CTA holds in registers
constexpr int kNormBwdCtas = 304;     // 2 x 152 SMs, of 256 threads: partial rows of dw

struct AddNormArgs {
  const void *x, *res;
  const float* weight;
  void *res_out, *y;
  float* scales;      // 8-bit output when non-null
  long long rows;
  int D;
  float eps;
};
struct AddNormBwdArgs {
  const void *dy, *sum, *dres;   // dres may be null
  const float* weight;
  void* dx;
  float *dw, *partial;
  long long rows;
  int D;
  float eps;
};
size_t add_rmsnorm_bwd_workspace_bytes(long long rows, int D);
cudaError_t launch_add_rmsnorm(const AddNormArgs& a, bool f32, cudaStream_t stream);
cudaError_t launch_add_rmsnorm_bwd(const AddNormBwdArgs& a, bool f32, cudaStream_t stream);

}  // namespace gdr
