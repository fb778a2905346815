// Norm after a block, gated and scaled residual sum, norm before the next
// block, in one pass over the rows:
//   p = y rstd(y) (w_post + off) or y;  r = x + s a(gate) p;  n = r rstd(r) (w_pre + off)
// with rstd(z) = 1/sqrt(mean z^2 + eps).  Everything between the loads and the
// stores is fp32; n is the norm of the unrounded r.
#include <atomic>

#include "norm.cuh"

namespace moe {
namespace {

template <typename XT, typename YT, bool VEC, int NV, bool PERCOL>
__global__ void __launch_bounds__(512) norm_fwd_kernel(const NormArgs a) {
  __shared__ alignas(16) float s_red[2][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.W, groups = (blockDim.x >> 5) / W;
  const int grp = warp / W, first = grp * W;
  const int v0 = (warp - first) * 32 + lane;  // share numbers v0 + i * 32 W
  const int d = a.d;
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const float inv_d = 1.f / static_cast<float>(d);
  int turn = 0;  // which of the two arrays the next row sum uses
  pdl_wait();
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < a.T;
       base += static_cast<int64_t>(gridDim.x) * groups) {
    const int64_t row = base + grp;
    const bool ok = row < a.T;
    const int64_t off = ok ? row * d : 0;
    const int dd = ok ? d : 0;  // no column of a row past the end
    float x[NV][8], y[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      Raw8<XT> rx;
      Raw8<YT> ry;
      load8<VEC>(static_cast<const XT*>(a.x) + off, v, a.x != nullptr ? dd : 0, rx);
      load8<VEC>(static_cast<const YT*>(a.y) + off, v, has_y ? dd : 0, ry);
      widen(rx, x[i]);
      widen(ry, y[i]);
    }
    if (has_y) {
      float rs = 1.f;
      if (post) {
        float sum[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[0] = fmaf(y[i][e], y[i][e], sum[0]);
        row_sum<1>(sum, s_red[turn], W, warp, first);
        turn ^= 1;
        rs = rsqrtf(fmaf(sum[0], inv_d, a.eps));
        if (ok && v0 == 0) a.rstd_y[row] = rs;
      }
      float fac = a.scale * rs;
      if (a.gate_kind == MOE_GATE_TOKEN) {
        float g, dg;
        gate_value(ok ? static_cast<const float*>(a.gate)[row] : 0.f, a.sigmoid, g, dg);
        fac *= g;
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * 32 * W;
        float w[8];
        if (post) {
          load8f<VEC>(a.w_post, v, d, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] *= w[e] + a.w_off;
        }
        if (PERCOL && a.gate_kind >= MOE_GATE_CHANNEL) {
          if (a.gate_kind == MOE_GATE_CHANNEL) {
            load8f<VEC>(static_cast<const float*>(a.gate), v, d, w);
          } else {
            Raw8<YT> rg;
            load8<VEC>(static_cast<const YT*>(a.gate) + off, v, dd, rg);
            widen(rg, w);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float g, dg;
            gate_value(w[e], a.sigmoid, g, dg);
            y[i][e] *= g;
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = fmaf(fac, y[i][e], x[i][e]);
        put8<XT, VEC>(static_cast<XT*>(a.r) + off, v, dd, x[i]);
      }
    }
    if (pre) {
      float sum[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(x[i][e], x[i][e], sum[0]);
      row_sum<1>(sum, s_red[turn], W, warp, first);
      turn ^= 1;
      const float rs = rsqrtf(fmaf(sum[0], inv_d, a.eps));
      if (ok && v0 == 0) a.rstd_r[row] = rs;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * 32 * W;
        float w[8];
        load8f<VEC>(a.w_pre, v, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] *= rs * (w[e] + a.w_off);
        put8<YT, VEC>(static_cast<YT*>(a.n) + off, v, dd, x[i]);
      }
    }
  }
}

template <typename XT, typename YT, bool VEC, int NV, bool PERCOL>
cudaError_t go(const NormArgs& a, cudaStream_t s) {
  const int groups = norm_groups(a.d), threads = groups * a.W * 32;
  // blocks that fit an SM, found once for each block size
  static std::atomic<int> fit[kNormMaxWarps + 1];
  int per = fit[threads / 32].load(std::memory_order_relaxed);
  if (per == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &per, norm_fwd_kernel<XT, YT, VEC, NV, PERCOL>, threads, 0);
    if (e != cudaSuccess) return e;
    if (per < 1) per = 1;
    fit[threads / 32].store(per, std::memory_order_relaxed);
  }
  const int64_t need = (a.T + groups - 1) / groups;
  const int64_t most = static_cast<int64_t>(per) * kSMs;
  return launch_pdl(norm_fwd_kernel<XT, YT, VEC, NV, PERCOL>,
                    dim3(static_cast<unsigned>(need < most ? need : most)), dim3(threads), 0, s, a);
}

template <typename XT, typename YT>
cudaError_t pick(const NormArgs& a, bool vec, cudaStream_t s) {
  const bool percol = a.gate_kind >= MOE_GATE_CHANNEL;
  switch (norm_nv(a.d)) {
    case 1:
      return !vec     ? go<XT, YT, false, 1, true>(a, s)
             : percol ? go<XT, YT, true, 1, true>(a, s)
                      : go<XT, YT, true, 1, false>(a, s);
    case 2:
      return !vec     ? go<XT, YT, false, 2, true>(a, s)
             : percol ? go<XT, YT, true, 2, true>(a, s)
                      : go<XT, YT, true, 2, false>(a, s);
    default:
      return !vec     ? go<XT, YT, false, 4, true>(a, s)
             : percol ? go<XT, YT, true, 4, true>(a, s)
                      : go<XT, YT, true, 4, false>(a, s);
  }
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int x_type, int y_type, bool vec, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (x_type == MOE_BF16) return pick<bf16_t, bf16_t>(a, vec, s);
  return y_type == MOE_BF16 ? pick<float, bf16_t>(a, vec, s) : pick<float, float>(a, vec, s);
}

}  // namespace moe
