// The norms after and before a block, with its gate and scale on the way into the residual:
//   u = x rsqrt(mean_c x^2 + eps) wa,   r = round(res + scale sigmoid(gate) u),
//   y = r rsqrt(mean_c r^2 + eps) wb,
// and the gradients, for dy of y and dres of r: with nx = x rsqrt(..), nr = r rsqrt(..),
//   dr = dres + rsqrt(mean r^2) (wb dy - nr mean_c(wb dy nr)),   dwb = sum_rows dy nr
//   dgate = dr scale wa nx sg (1 - sg),   m = sum_rows dr sg nx: dscale = wa m, dwa = scale m
//   dx = rsqrt(mean x^2) (t - nx mean_c(t nx)),  t = dr scale wa sg.
// scale and wa enter as one product, rounded to fp32 once.
//
// Streams bound by HBM: every row is read once and stays in registers through its two
// sums. A row is spread over TPR threads, one or two vectors of 8 columns each; the CTAs
// are persistent, walk the rows and request the next row's vectors before the current
// row's sums, so that loads are in flight through the barriers. 65536 x 4096 bf16: 396 us, all
// of measured HBM (462 with an exact division in the sigmoid); gradients of 16384 x 2048: 94
// us, 0.84, of which 6 are the second launch.
#include "block_norms.h"

#include <type_traits>

#include "column_sum.cuh"
#include "pair.cuh"
#include "vec_io.cuh"

namespace gdr {
namespace {

constexpr int kBwdCtas = 304;    // 2 x 152 SMs, of 256 threads: partial rows of the weights

template <typename T>
__device__ __forceinline__ float rounded(float x) {
  return static_cast<float>(static_cast<T>(x));
}

// 8 elements as pairs, and back with one rounding.
template <typename T>
__device__ __forceinline__ void pairs(const Raw8<T>& r, f32x2 (&x)[4]) {
  float f[8];
  r.get(f);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pair(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void store_pairs(T* p, const f32x2 (&x)[4]) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) split(x[i], f[2 * i], f[2 * i + 1]);
  store8(p, f);
}

// Sums of two values over the TPR threads of a row; `red` has a slot per warp, and
// consecutive calls take different ones of its parts, so one barrier each is enough.
template <int TPR>
__device__ __forceinline__ void row_sum(float& x, float& y, float2 (&red)[16]) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    x += __shfl_xor_sync(0xffffffffu, x, off);
    y += __shfl_xor_sync(0xffffffffu, y, off);
  }
  if (TPR > 32) {
    const int warp = threadIdx.x >> 5, first = warp & ~(TPR / 32 - 1);
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(x, y);
    __syncthreads();
    x = y = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      const float2 v = red[first + i];
      x += v.x;
      y += v.y;
    }
  }
}

template <int TPR>
constexpr int threads() { return TPR > 32 ? TPR : 256; }

// The columns' constants: post * scale and pre.
template <int TPR, int VEC>
__device__ __forceinline__ void load_weights(const float* post, const float* scale,
                                             const float* pre, int lane, int nv,
                                             float (&ws)[VEC][8], float (&wp)[VEC][8]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
    float s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      ws[i][j] = wp[i][j] = 0.f;
      s[j] = 1.f;
    }
    if (c < nv) {
      load8(post + 8 * c, ws[i]);
      load8(pre + 8 * c, wp[i]);
      if (scale) load8(scale + 8 * c, s);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ws[i][j] *= s[j];
  }
}

template <typename T, int TPR, int VEC>
__global__ void __launch_bounds__(threads<TPR>(), sizeof(T) == 2 ? 512 / threads<TPR>() : 1)
    block_norms_kernel(const BlockNormsArgs a) {
  constexpr int kRows = threads<TPR>() / TPR;
  __shared__ float2 red[2][16];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nv = a.D / 8;
  float ws[VEC][8], wp[VEC][8];
  Raw8<T> rx[VEC], rg[VEC], rr[VEC];
  auto fetch = [&](long long row) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      rg[i].zero();
      if (row < a.rows && c < nv) {
        rx[i].load(static_cast<const T*>(a.x) + row * a.D + 8 * c);
        if (a.gate) rg[i].load(static_cast<const T*>(a.gate) + row * a.D + 8 * c);
        rr[i].load(static_cast<const T*>(a.residual) + row * a.D + 8 * c);
      } else {
        rx[i].zero();
        rr[i].zero();
      }
    }
  };
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  long long r0 = static_cast<long long>(blockIdx.x) * kRows;
  fetch(r0 + sub);
  load_weights<TPR, VEC>(a.post, a.scale, a.pre, lane, nv, ws, wp);
  const float n = static_cast<float>(a.D);
  for (; r0 < a.rows; r0 += step) {
    const long long row = r0 + sub;
    const bool live = row < a.rows;
    float v[VEC][8], ss = 0.f, none = 0.f;
    Raw8<T> kg[VEC], kr[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      rx[i].get(v[i]);
      kg[i] = rg[i];
      kr[i] = rr[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    fetch(row + step);
    row_sum<TPR>(ss, none, red[0]);
    const float ix = rsqrtf(ss / n + a.eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      float g[8], r[8];
      kg[i].get(g);
      kr[i].get(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float u = v[i][j] * ix * ws[i][j];
        if (a.gate) u *= sigmoid(g[j]);
        v[i][j] = rounded<T>(r[j] + u);
        ss = fmaf(v[i][j], v[i][j], ss);
      }
      if (live && c < nv) store8(static_cast<T*>(a.residual_out) + row * a.D + 8 * c, v[i]);
    }
    row_sum<TPR>(ss, none, red[1]);
    const float ir = rsqrtf(ss / n + a.eps);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * ir * wp[i][j];
      if (live && c < nv) store8(static_cast<T*>(a.y) + row * a.D + 8 * c, v[i]);
    }
  }
}

// 16 bytes at a time from global to shared memory.
template <typename T>
__device__ __forceinline__ void copy8(uint4* to, const T* from) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + i)),
                 "l"(reinterpret_cast<const uint4*>(from) + i)
                 : "memory");
}

// Rows on their way or in use: the inputs are copied to the thread's own places in shared
// memory, which takes no registers and no barrier. One row ahead; two ahead take as long or
// longer (65536 x 512 bf16: 100 us for 87). Of more than 4096 columns the next row is requested
// as soon as the current one is in registers, into its places (4096 x 8192 bf16: 103 us, 115
// with places for two rows, 159 in registers, which spilled).
constexpr int kInputs = 5;      // sum, dy, dres, x, gate
template <int VEC>
constexpr int stages() { return VEC == 1 ? 2 : 1; }

// Each thread keeps its columns' sums in registers over all its rows; the CTA's row groups
// add theirs at the end, in a fixed order, to one row of `partial` ([2, D]: m and dpre).
template <typename T, int TPR, int VEC>
__global__ void __launch_bounds__(threads<TPR>(), sizeof(T) == 2 ? 512 / threads<TPR>() : 1)
    block_norms_bwd_kernel(const BlockNormsBwdArgs a) {
  constexpr int kThreads = threads<TPR>(), kRows = kThreads / TPR;
  constexpr int kStages = stages<VEC>(), kWords = sizeof(T) / 2;
  extern __shared__ __align__(16) unsigned char raw_smem[];
  uint4* ring = reinterpret_cast<uint4*>(raw_smem);   // [stage][input][vector][thread][kWords]
  __shared__ float2 red[2][16];
  __shared__ float sums[kRows > 1 ? kThreads * 8 : 1];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int nv = a.D / 8;
  f32x2 ws[VEC][4], wp[VEC][4], dm[VEC][4], dp[VEC][4];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) dm[i][j] = dp[i][j] = 0;
  const T* const in[kInputs] = {static_cast<const T*>(a.sum), static_cast<const T*>(a.dy),
                                static_cast<const T*>(a.dres), static_cast<const T*>(a.x),
                                static_cast<const T*>(a.gate)};
  auto place = [&](int stage, int k, int i) {
    return ring + (((stage * kInputs + k) * VEC + i) * kThreads + threadIdx.x) * kWords;
  };
  // what is not there stays zero: columns past D, a missing dres or gate
#pragma unroll
  for (int st = 0; st < kStages; ++st)
#pragma unroll
    for (int k = 0; k < kInputs; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int w = 0; w < kWords; ++w) place(st, k, i)[w] = make_uint4(0u, 0u, 0u, 0u);
  auto fetch = [&](int stage, long long row) {
    if (row < a.rows)
#pragma unroll
      for (int k = 0; k < kInputs; ++k)
        if (in[k])
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const int c = lane + i * TPR;
            if (c < nv) copy8(place(stage, k, i), in[k] + row * a.D + 8 * c);
          }
    if (kRows > 1 && row >= a.rows)      // beside the last rows: zeros
#pragma unroll
      for (int k = 0; k < kInputs; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
#pragma unroll
          for (int w = 0; w < kWords; ++w) place(stage, k, i)[w] = make_uint4(0u, 0u, 0u, 0u);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto get = [&](int stage, int k, int i, f32x2 (&v)[4]) {
    Raw8<T> r;
    const uint4* p = place(stage, k, i);
#pragma unroll
    for (int w = 0; w < kWords; ++w) r.u[w] = p[w];
    pairs(r, v);
  };
  const long long step = static_cast<long long>(gridDim.x) * kRows;
  const long long first = static_cast<long long>(blockIdx.x) * kRows;
#pragma unroll
  for (int st = 0; st < (kStages > 1 ? kStages - 1 : 1); ++st) fetch(st, first + sub + st * step);
  {
    float s[VEC][8], p[VEC][8];
    load_weights<TPR, VEC>(a.post, a.scale, a.pre, lane, nv, s, p);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ws[i][j] = pair(s[i][2 * j], s[i][2 * j + 1]);
        wp[i][j] = pair(p[i][2 * j], p[i][2 * j + 1]);
      }
  }
  const float n = static_cast<float>(a.D);
  int stage = 0;
  for (long long r0 = first; r0 < a.rows; r0 += step) {
    const long long row = r0 + sub;
    const bool live = row < a.rows;
    if (kStages > 1) {
      const int next = stage == 0 ? kStages - 1 : stage - 1;
      fetch(next, row + (kStages - 1) * step);
    }
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    f32x2 ss = 0, dot = 0, xx = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      f32x2 r[4], dy[4];
      get(stage, 0, i, r);
      get(stage, 1, i, dy);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        ss = fma2(r[j], r[j], ss);
        dot = fma2(mul2(wp[i][j], dy[j]), r[j], dot);
      }
    }
    // (what waits for no sum, ahead of the first)
    f32x2 dr[VEC][4], sg[VEC][4], x[VEC][4];
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      get(stage, 3, i, x[i]);
      get(stage, 4, i, sg[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) xx = fma2(x[i][j], x[i][j], xx);
      if (a.gate) {
#pragma unroll
        for (int j = 0; j < 4; ++j) sg[i][j] = sigmoid2(sg[i][j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) sg[i][j] = both(1.f);
      }
    }
    float s0 = sum2(ss), s1 = sum2(dot);
    row_sum<TPR>(s0, s1, red[0]);
    // (zero for a row that is not there, which then adds nothing: with eps = 0 its zeros would
    // have no finite norm)
    const float ir = kRows == 1 || live ? rsqrtf(s0 / n + a.eps) : 0.f;
    const f32x2 ir2 = both(ir), mr = both(-ir * ir * (s1 / n));
    dot = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      f32x2 r[4], dy[4];
      get(stage, 0, i, r);
      get(stage, 1, i, dy);
      get(stage, 2, i, dr[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dp[i][j] = fma2(dy[j], mul2(r[j], ir2), dp[i][j]);
        dr[i][j] = fma2(ir2, fma2(wp[i][j], dy[j], mul2(r[j], mr)), dr[i][j]);
        dot = fma2(mul2(mul2(dr[i][j], ws[i][j]), sg[i][j]), x[i][j], dot);
      }
      if (live && c < nv) store_pairs(static_cast<T*>(a.dresidual) + row * a.D + 8 * c, dr[i]);
    }
    if (kStages == 1) fetch(0, row + step);
    s0 = sum2(xx);
    s1 = sum2(dot);
    row_sum<TPR>(s0, s1, red[1]);
    const float ix = kRows == 1 || live ? rsqrtf(s0 / n + a.eps) : 0.f;
    const f32x2 ix2 = both(ix), mx = both(-ix * ix * (s1 / n));
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      f32x2 dx[4], dg[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 nx = mul2(x[i][j], ix2), d = mul2(dr[i][j], sg[i][j]), t = mul2(d, ws[i][j]);
        dm[i][j] = fma2(d, nx, dm[i][j]);
        dg[j] = mul2(mul2(t, nx), fma2(sg[i][j], both(-1.f), both(1.f)));
        dx[j] = mul2(ix2, fma2(x[i][j], mx, t));
      }
      if (!(live && c < nv)) continue;
      store_pairs(static_cast<T*>(a.dx) + row * a.D + 8 * c, dx);
      if (a.gate) store_pairs(static_cast<T*>(a.dgate) + row * a.D + 8 * c, dg);
    }
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
#pragma unroll
  for (int part = 0; part < 2; ++part)
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      float s[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(part ? dp[i][j] : dm[i][j], s[2 * j], s[2 * j + 1]);
      if constexpr (kRows > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[threadIdx.x * 8 + j] = s[j];
        __syncthreads();
        if (sub == 0)
          for (int r = 1; r < kRows; ++r)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += sums[(r * TPR + lane) * 8 + j];
      }
      if (sub == 0 && c < nv) {
        float4* p = reinterpret_cast<float4*>(
            a.partial + (static_cast<size_t>(blockIdx.x) * 2 + part) * a.D + 8 * c);
        p[0] = make_float4(s[0], s[1], s[2], s[3]);
        p[1] = make_float4(s[4], s[5], s[6], s[7]);
      }
    }
}

__global__ void __launch_bounds__(1024) block_weights_kernel(const BlockNormsBwdArgs a, int rows) {
  column_sum<32>(a.partial, rows, 2 * a.D, [&](int i, float s) {
    if (i >= a.D) {
      a.dpre[i - a.D] = s;
    } else {
      a.dpost[i] = a.scale ? s * a.scale[i] : s;
      if (a.scale) a.dscale[i] = s * a.post[i];
    }
  });
}

// Threads per row and vectors per thread for a row of D columns. Two vectors a thread where
// registers allow: fewer threads wait for a row's sums (forward, 65536 x 4096 bf16: 551 us
// with one). The backward has five inputs and two sums a column (16384 x 2048: 255 us with
// two, which spill).
template <int VEC, class F>
cudaError_t by_width(int D, F f) {
  const int nv = D / 8;
  using std::integral_constant;
  if (nv <= 32) return f(integral_constant<int, 32>{}, integral_constant<int, 1>{});
  if (nv <= 32 * VEC) return f(integral_constant<int, 32>{}, integral_constant<int, VEC>{});
  if (nv <= 64 * VEC) return f(integral_constant<int, 64>{}, integral_constant<int, VEC>{});
  if (nv <= 128 * VEC) return f(integral_constant<int, 128>{}, integral_constant<int, VEC>{});
  if (nv <= 256 * VEC) return f(integral_constant<int, 256>{}, integral_constant<int, VEC>{});
  if (nv <= 512 * VEC) return f(integral_constant<int, 512>{}, integral_constant<int, VEC>{});
  return f(integral_constant<int, 512>{}, integral_constant<int, 2>{});
}

int ctas(long long rows, int per_cta, int most) {
  const long long want = (rows + per_cta - 1) / per_cta;
  return static_cast<int>(want < most ? want : most);
}

// CTAs of a kernel that all SMs hold at once, asked for once per device.
template <auto Kern>
int resident(int threads) {
  constexpr int kMaxDevices = 64;
  static int held[kMaxDevices] = {};
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices) return 1;
  if (held[dev] == 0 &&
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, Kern, threads, 0) == cudaSuccess)
    held[dev] = sms * per;
  return held[dev] > 0 ? held[dev] : 1;
}

template <typename T>
cudaError_t fwd(const BlockNormsArgs& a, cudaStream_t stream) {
  return by_width<2>(a.D, [&](auto tpr, auto vec) {
    constexpr int kThreads = threads<tpr>(), kRows = kThreads / tpr;
    const int grid = ctas(a.rows, kRows, resident<block_norms_kernel<T, tpr, vec>>(kThreads));
    block_norms_kernel<T, tpr, vec><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
  });
}

template <typename T>
cudaError_t bwd(const BlockNormsBwdArgs& a, cudaStream_t stream) {
  return by_width<1>(a.D, [&](auto tpr, auto vec) {
    constexpr int kThreads = threads<tpr>(), kRows = kThreads / tpr;
    const int grid = ctas(a.rows, kRows, kBwdCtas * 256 / kThreads);
    constexpr int kBytes = stages<vec>() * kInputs * vec * 8 * sizeof(T) * kThreads;
    const cudaError_t err = cudaFuncSetAttribute(block_norms_bwd_kernel<T, tpr, vec>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (err != cudaSuccess) return err;
    block_norms_bwd_kernel<T, tpr, vec><<<grid, kThreads, kBytes, stream>>>(a);
    block_weights_kernel<<<(2 * a.D + 31) / 32, 1024, 0, stream>>>(a, grid);
    return cudaGetLastError();
  });
}

}  // namespace

size_t block_norms_bwd_workspace_bytes(long long rows, int D) {
  size_t bytes = 0;
  by_width<1>(D, [&](auto tpr, auto) {
    constexpr int kThreads = threads<tpr>(), kRows = kThreads / tpr;
    bytes = static_cast<size_t>(ctas(rows, kRows, kBwdCtas * 256 / kThreads)) * 2 * D *
            sizeof(float);
    return cudaSuccess;
  });
  return bytes;
}

cudaError_t launch_block_norms(const BlockNormsArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? fwd<float>(a, stream) : fwd<__nv_bfloat16>(a, stream);
}
cudaError_t launch_block_norms_bwd(const BlockNormsBwdArgs& a, bool f32, cudaStream_t stream) {
  return f32 ? bwd<float>(a, stream) : bwd<__nv_bfloat16>(a, stream);
}

}  // namespace gdr
