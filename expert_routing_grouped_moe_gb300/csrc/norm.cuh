// Kernels of the norms around a block, forward and backward (norm_fwd.cu,
// norm_bwd.cu): what the two share.
#pragma once

#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "rowvec.cuh"

namespace moe {

struct NormArgs {
  const void* x;      // fwd: residual stream, bwd: dr       [T,d] residual type
  const void* y;      // block output                        [T,d] block type
  const void* gate;   // TOKEN [T], CHANNEL [d] fp32; ELEMENT [T,d] block type
  const float* w_post;
  const float* w_pre;
  void* r;            // fwd: out; bwd: the saved r          [T,d] residual type
  void* n;            // fwd: out; bwd: dn                   [T,d] block type
  float* rstd_y;
  float* rstd_r;
  void* dx;           // bwd outputs
  void* dy;
  void* dgate;
  float* part;        // bwd: column partial sums [rows of partials][nsum][d]
  int sum_post, sum_pre, sum_gate;  // index of each column sum in part, -1: not wanted
  int nsum;
  int64_t T;
  int d, W;           // columns; warps that share a row
  int gate_kind, sigmoid;
  float scale, eps, w_off;
};

// A row's shares: NV of 8 values for each thread of W warps, 32 W NV 8 >= d.
// The fewest values per thread whose row fits 16 warps, so that a row's loads
// are spread over as many threads as there are.
constexpr int kNormMaxWarps = 16;
constexpr int kNormMaxD = kNormMaxWarps * 32 * 8 * 4;
inline int norm_nv(int d) { return d <= 4096 ? 1 : d <= 8192 ? 2 : 4; }
inline int norm_warps(int d) { const int per = 256 * norm_nv(d); return (d + per - 1) / per; }
inline int norm_groups(int d) { const int w = norm_warps(d); return w >= 8 ? 1 : 8 / w; }

// Sums v over the W warps of this thread's row group (all threads of the block
// call it, same W).  buf: two arrays of 32 warps x 4; the caller alternates
// them, so one barrier per call is enough: a warp writes an array again only
// after the barrier of the call in between, which every reader has passed.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*buf)[4], int W, int warp,
                                        int first) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < K; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  if (W == 1) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < K; ++i) buf[warp][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < K; ++i) v[i] = 0.f;
  for (int w = 0; w < W; ++w) {
    const float4 q = *reinterpret_cast<const float4*>(buf[first + w]);
    v[0] += q.x;
    if (K > 1) v[1] += q.y;
    if (K > 2) v[2] += q.z;
  }
}

// a(gate) and its derivative.
__device__ __forceinline__ void gate_value(float g, int sigmoid, float& a, float& da) {
  if (sigmoid) {
    a = 1.f / (1.f + expf(-g));
    da = a * (1.f / (1.f + expf(g)));  // 1 - a without its cancellation
  } else {
    a = g;
    da = 1.f;
  }
}

cudaError_t launch_norm_fwd(const NormArgs& a, int x_type, int y_type, bool vec, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, int x_type, int y_type, bool vec, int blocks,
                            float* const (&sums)[3], cudaStream_t s);

}  // namespace moe
