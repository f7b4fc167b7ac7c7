// Launch interface of the state space recurrence (state_space*.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr {

// Pointers as documented in include/gdr.h. Strides are elements between tokens.
struct SpaceArgs {
  const void *x, *dt, *z, *Bm, *Cm, *dy;
  const float *A, *skip, *dt_bias, *h0, *dhT;
  const unsigned char* starts;
  void *y, *dx, *ddt, *dz, *dBm, *dCm;
  float *hT, *dA, *dskip, *ddt_bias, *dh0;
  int B, T, D, G, N;
  bool softplus;
  long long xs, dts, zs, bs, cs;
};

constexpr int kSpaceTile = 16;     // tokens between the backward's kept states

// One call's cut of the sequences: `segments` runs of `seg_len` tokens (whole tiles; the
// last may be shorter) and the workspace's arrays, all fp32.
struct SpaceSplit {
  int segments = 1;
  int seg_len = 0;
  int tiles = 0;              // backward: tiles of kSpaceTile tokens in a sequence
  int blocks = 1;             // backward: CTAs over the channels (dBm's and dCm's partial sums)
  // slot 0: h0; slot 1: the state behind segment 0; slot s > 1: what segment s - 1 alone adds,
  // after the chain the state entering segment s
  float* h = nullptr;         // [B, segments, D, N]
  float* total = nullptr;     // [B, segments, D] a segment's sum of u
  int* cleared = nullptr;     // [B, segments] nonzero: a document starts in it
  // backward: slot S - 1: dhT; slot s < S - 1: the gradient that segment s + 1 passes on
  // (alone; the last segment's with dhT's), after the chain all that enters segment s
  float* e = nullptr;         // [B, segments, D, N]
  float* kept = nullptr;      // [B, tiles, D, N] a segment's own state entering each tile
  float* kept_sum = nullptr;  // [B, tiles, D] the segment's sum of u up to there
  int* kept_clear = nullptr;  // [B, tiles] nonzero: a document started since the segment did
  float* dA_part = nullptr;   // [B * segments, D, N]
  float* d_part = nullptr;    // [B * segments, 2, D] of dskip and ddt_bias
  float* bc_part = nullptr;   // [blocks, B, T, G, 2, N] of dBm and dCm
};

int space_channels(int N, bool narrow);   // channels of a CTA: forward, backward
int space_bwd_channels(int N, bool f32);
cudaError_t launch_space_states(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                                cudaStream_t stream);
cudaError_t launch_space_chain(const SpaceArgs& a, const SpaceSplit& sp, bool backward,
                               cudaStream_t stream);
cudaError_t launch_space_walk(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                              cudaStream_t stream);
cudaError_t launch_space_bwd_states(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                                    cudaStream_t stream);
cudaError_t launch_space_bwd(const SpaceArgs& a, const SpaceSplit& sp, bool f32,
                             cudaStream_t stream);
cudaError_t launch_space_step(const SpaceArgs& a, bool f32, cudaStream_t stream);

}  // namespace gdr
