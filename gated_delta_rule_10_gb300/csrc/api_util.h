// Small helpers of the C ABI's argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "gdr.h"

namespace gdr {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline bool given16(const void* p) { return p && aligned(p, 16); }
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline gdr_status status_of(cudaError_t err) { return err == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }
inline cudaStream_t stream_of(gdr_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
inline gdr_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return GDR_OK;
  if (!ws || have < need) return GDR_ERR_WORKSPACE;
  return aligned(ws, 16) ? GDR_OK : GDR_ERR_INVALID_ARG;
}
// No output is an input's or another output's buffer (those that are there). Only equal
// addresses are seen: callers keep the rest of what they were asked for.
inline bool apart(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (const void* const* o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void* i : ins)
      if (i == *o) return false;
    for (const void* const* q = outs.begin(); q != o; ++q)
      if (*q == *o) return false;
  }
  return true;
}

}  // namespace gdr
