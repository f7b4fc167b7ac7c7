// Launch interface of the rotary positions (rotary.cu).
#pragma once

#include <cuda_runtime.h>

namespace gdr {

struct RotaryArgs {
  const void *q, *k;
  void *q_out, *k_out;
  const float *cos_t, *sin_t;   // [table_len, rot / 2]
  const int* pos;               // [tokens], or null: start + token % T
  long long tokens;
  int T, H, Hk, d, rot, start, table_len;
  long long sq, sk, sqo, sko;   // elements between tokens
  bool interleaved, inverse, copy_tail;
};
cudaError_t launch_rotary(const RotaryArgs& a, bool f32, cudaStream_t stream);

struct RotaryTableArgs {
  float *cos_t, *sin_t;
  int len, rot, kind;
  double base, factor, original, fast, slow, magnitude;
};
cudaError_t launch_rotary_table(const RotaryTableArgs& a, cudaStream_t stream);

}  // namespace gdr
