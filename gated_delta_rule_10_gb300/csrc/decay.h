// Launch interface of the linear attention with a decay for each head
// (layer_api.cu and the kernels behind it).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>

namespace gdr {

// Pointers and sizes as documented in include/gdr.h. Strides are elements
// between consecutive tokens; a head's channels are dense and head h of q and k
// starts at (h / (H / Hk)) * dk.
struct DecayArgs {
  const void *q, *k, *v, *dO;
  const float *g, *h0, *dhT;
  void *o, *dq, *dk, *dv;
  float *hT, *dg, *dh0;
  int B, T, H, Hk, nk, nv;      // nk, nv: key and value widths
  long long sq, sk, sv;
  bool per_head;                // g is [H] instead of [B, T, H]
  float scale;
};

// One call's cut of the sequences: `segments` runs of `seg_len` tokens (whole
// chunks; the last may be shorter), each of `parts_per` pieces of `piece_len`
// tokens whose own states are computed separately (`pieces` in all), and the
// workspace's arrays. States are [B * H, slots, nk, nv] fp32.
struct DecaySplit {
  int segments = 1;
  int seg_len = 0;
  int pieces = 1, parts_per = 1, piece_len = 0;
  int slots = 0;              // state slots per (batch, head): pieces, backward + 1
  int parts = 1;              // partial sums of each boundary dot product
  float* S = nullptr;         // slot p: the state entering piece p
  float* D = nullptr;         // slot p: the gradient of that state (backward)
  float* decay = nullptr;     // [B * H, pieces] a piece's decay (decay_code)
  float* dots = nullptr;      // [B * H, slots, parts] partial <S_p, D_p>
  int firsts = 1;             // partial sums of the same product at the sequence's start,
  float* first = nullptr;     // [B * H, firsts] <h0, D_0> from the walk that gives dk
  // Terms of the gate's gradient by token, [flows, B * H, T] (the parts add up):
  // what its row takes from before its block of 32 tokens, what its keys and values
  // give to after it, and [nears, B * H, T] the difference within the block.
  int flows = 1, nears = 1;
  float* from = nullptr;
  float* to = nullptr;
  float* near = nullptr;
  float* dq_part = nullptr;   // [B, T, H, nk] per-head gradients of shared q, k
  float* dk_part = nullptr;
  float* dg_part = nullptr;   // [B * H, segments] sums for a per-head decay
  // slot of the state entering segment p (p = segments: leaving the last)
  __host__ __device__ int slot_of(int p) const { return p < segments ? p * parts_per : pieces; }
  // pieces whose own state is needed: up to the last segment's start, or to the end
  __host__ __device__ int states(bool to_end) const { return to_end ? pieces : slot_of(segments - 1); }
};

// A log-decay at or below this clears the state: exp() of it is zero in fp32.
constexpr float kDecayReset = -104.f;

#ifdef __CUDACC__
// The decay e^x of a state over a chunk or a piece, and its use. Between 1/2 and 1 it is
// kept as its distance from 1 (sign set): a fixed decay's rounding is the same in every
// chunk, and over the chunks that a slow decay reaches it adds up (4.6e-6 of 64 bits for
// 8192 tokens in fp32; so kept 2.6e-7).
__device__ __forceinline__ float decay_code(float x) {
  return x > -0.693f && x <= 0.f ? -fabsf(expm1f(x)) : expf(x);
}
__device__ __forceinline__ float decayed(float code, float s, float add) {
  return signbit(code) ? fmaf(code, s, s + add) : fmaf(code, s, add);
}
#endif

// fp32 inputs: split-tf32 warp products, chunks of 64 tokens (decay_f32.cu).
cudaError_t launch_decay_states_f32(const DecayArgs& a, const DecaySplit& sp, bool reverse,
                                    cudaStream_t stream);
cudaError_t launch_decay_fwd_f32(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream);
cudaError_t launch_decay_bwd_f32(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream);
// bf16 inputs on tcgen05, chunks of 128 tokens (decay_tc.cu).
cudaError_t launch_decay_states_tc(const DecayArgs& a, const DecaySplit& sp, bool reverse,
                                   cudaStream_t stream);
cudaError_t launch_decay_fwd_tc(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream);
cudaError_t launch_decay_bwd_tc(const DecayArgs& a, const DecaySplit& sp, cudaStream_t stream);
// Chains the pieces' states (decay_chain.cu); backward also chains the
// states' gradients and writes the boundary dot products.
cudaError_t launch_decay_chain(const DecayArgs& a, const DecaySplit& sp, bool backward,
                               cudaStream_t stream);
// The gate's gradient from the flow terms, and the sums over shared heads.
cudaError_t launch_decay_gate_grad(const DecayArgs& a, const DecaySplit& sp, bool f32,
                                   cudaStream_t stream);

struct DecayStepArgs {
  const void *q, *k, *v;
  const float* g;
  float* state;
  void* o;
  int N, H, Hk;
  long long sq, sk, sv;
  bool per_head;
  float scale;
};
cudaError_t launch_decay_step(const DecayStepArgs& a, int nk, int nv, bool f32,
                              cudaStream_t stream);

}  // namespace gdr
