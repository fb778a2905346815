// Backward of norm_fwd.cu, in one pass over the rows.  With rh = r rstd_r,
// yh = y rstd_y, u = w_pre + off, q = w_post + off:
//   e = dr + rstd_r dn u,  c1 = mean(dn u rh),  t = e - rstd_r c1 rh        dx = t
//   p = yh q (or y);  dp = s a t;  dy = rstd_y (dp q - yh mean(dp p))      (or dp)
//   dgate = s a' t p, summed over what the gate is broadcast over
//   dw_pre = sum_rows dn rh;  dw_post = sum_rows dp yh
// t is linear in c1, so one reduction gives every row sum:
//   S1 = sum dn u rh,  S2 = sum A p e,  S3 = sum A p rh,
//   sum A p t = S2 - rstd_r c1 S3     (A = a(gate) where it varies along the row, else 1)
// Column sums are kept in registers over the rows of a block, written once as
// partials and added by a second kernel in a fixed order (no atomics).
#include <atomic>

#include "norm.cuh"

namespace moe {
namespace {

template <typename XT, typename YT, bool VEC, int NV, bool PERCOL, bool SUMS>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const NormArgs a) {
  __shared__ alignas(16) float s_red[2][32][4];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.W, groups = (blockDim.x >> 5) / W;
  const int grp = warp / W, first = grp * W;
  const int v0 = (warp - first) * 32 + lane;
  const int d = a.d;
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const bool sum_gate_row = a.gate_kind == MOE_GATE_TOKEN && a.dgate != nullptr;
  const float inv_d = 1.f / static_cast<float>(d);
  float acc_post[NV][8], acc_pre[NV][8], acc_gate[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc_post[i][e] = acc_pre[i][e] = acc_gate[i][e] = 0.f;
  int turn = 0;
  pdl_wait();
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * groups; base < a.T;
       base += static_cast<int64_t>(gridDim.x) * groups, turn ^= 1) {
    const int64_t row = base + grp;
    const bool ok = row < a.T;
    const int64_t off = ok ? row * d : 0;
    const int dd = ok ? d : 0;
    Raw8<XT> rdr[NV], rr[NV];
    Raw8<YT> rdn[NV], ry[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      load8<VEC>(static_cast<const XT*>(a.x) + off, v, a.x != nullptr ? dd : 0, rdr[i]);
      load8<VEC>(static_cast<const XT*>(a.r) + off, v, pre ? dd : 0, rr[i]);
      load8<VEC>(static_cast<const YT*>(a.n) + off, v, pre ? dd : 0, rdn[i]);
      load8<VEC>(static_cast<const YT*>(a.y) + off, v, has_y ? dd : 0, ry[i]);
    }
    const float rs_r = pre && ok ? a.rstd_r[row] : 0.f;
    const float rs_y = post && ok ? a.rstd_y[row] : 0.f;
    float a_row = 1.f, da_row = 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN)
      gate_value(ok ? static_cast<const float*>(a.gate)[row] : 0.f, a.sigmoid, a_row, da_row);
    // pass 1: e in place of dr, rh in place of r; the row sums
    float ev[NV][8], rh[NV][8], ga[NV][8], gd[NV][8];
    float sum[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      widen(rdr[i], ev[i]);
      widen(rr[i], rh[i]);
      float dn[8], w[8];
      widen(rdn[i], dn);
      if (pre) {
        load8f<VEC>(a.w_pre, v, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          rh[i][e] *= rs_r;
          if (SUMS) acc_pre[i][e] = fmaf(dn[e], rh[i][e], acc_pre[i][e]);
          const float g = dn[e] * (w[e] + a.w_off);
          ev[i][e] = fmaf(rs_r, g, ev[i][e]);
          sum[0] = fmaf(g, rh[i][e], sum[0]);
        }
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
        for (int e = 0; e < 8; ++e) gate_value(w[e], a.sigmoid, ga[i][e], gd[i][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) ga[i][e] = 1.f;
      }
      if (post || sum_gate_row) {
        float y[8];
        widen(ry[i], y);
        if (post) load8f<VEC>(a.w_post, v, d, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = post ? y[e] * rs_y * (w[e] + a.w_off) : y[e];
          const float ap = ga[i][e] * p;
          sum[1] = fmaf(ap, ev[i][e], sum[1]);
          sum[2] = fmaf(ap, rh[i][e], sum[2]);
        }
      }
    }
    if (pre || post || sum_gate_row) row_sum<3>(sum, s_red[turn], W, warp, first);
    const float c1 = rs_r * sum[0] * inv_d;
    const float apt = sum[1] - c1 * sum[2];  // sum A p t
    if (sum_gate_row && ok && v0 == 0)
      static_cast<float*>(a.dgate)[row] = a.scale * da_row * apt;
    const float fac = a.scale * a_row;       // dp = fac A t
    const float c2 = fac * apt * inv_d;
    // pass 2: the outputs
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      float y[8], w[8], o[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) ev[i][e] = fmaf(-c1, rh[i][e], ev[i][e]);  // t
      put8<XT, VEC>(static_cast<XT*>(a.dx) + off, v, a.dx != nullptr ? dd : 0, ev[i]);
      if (!has_y) continue;
      widen(ry[i], y);
      if (post) load8f<VEC>(a.w_post, v, d, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dp = fac * ga[i][e] * ev[i][e];
        const float yh = y[e] * rs_y;
        const float q = post ? w[e] + a.w_off : 1.f;
        o[e] = post ? rs_y * fmaf(-yh, c2, dp * q) : dp;
        if (SUMS && post) acc_post[i][e] = fmaf(dp, yh, acc_post[i][e]);
        if (PERCOL) w[e] = a.scale * gd[i][e] * ev[i][e] * (post ? yh * q : y[e]);  // dgate
      }
      put8<YT, VEC>(static_cast<YT*>(a.dy) + off, v, a.dy != nullptr ? dd : 0, o);
      if (PERCOL && a.dgate != nullptr && a.gate_kind >= MOE_GATE_CHANNEL) {
        if (a.gate_kind == MOE_GATE_ELEMENT) {
          put8<YT, VEC>(static_cast<YT*>(a.dgate) + off, v, dd, w);
        } else if (SUMS) {
#pragma unroll
          for (int e = 0; e < 8; ++e) acc_gate[i][e] += ok ? w[e] : 0.f;
        }
      }
    }
  }
  if (!SUMS) return;
  float* part = a.part + (static_cast<int64_t>(blockIdx.x) * groups + grp) * a.nsum * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * 32 * W;
    if (a.sum_post >= 0) put8<float, VEC>(part + static_cast<int64_t>(a.sum_post) * d, v, d, acc_post[i]);
    if (a.sum_pre >= 0) put8<float, VEC>(part + static_cast<int64_t>(a.sum_pre) * d, v, d, acc_pre[i]);
    if (a.sum_gate >= 0) put8<float, VEC>(part + static_cast<int64_t>(a.sum_gate) * d, v, d, acc_gate[i]);
  }
}

// out_q[c] = sum over the P rows of partials of part[row][q][c], in row order
// within each of 8 interleaved sums, those added in order.
struct SumOuts {
  float* p[3];
};
__global__ void __launch_bounds__(256) norm_colsum_kernel(const float* part, int P, int nsum, int d,
                                                          SumOuts outs) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = static_cast<int64_t>(nsum) * d;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  pdl_wait();
  float t = 0.f;
  if (c < n) {
#pragma unroll 8
    for (int r = w; r < P; r += 8) t += part[r * n + c];
  }
  s[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < n) {
#pragma unroll
    for (int i = 1; i < 8; ++i) t += s[i][lane];
    const int q = static_cast<int>(c / d);
    outs.p[q][c - static_cast<int64_t>(q) * d] = t;
  }
}

template <typename XT, typename YT, bool VEC, int NV, bool PERCOL, bool SUMS>
cudaError_t go(const NormArgs& a, int blocks, cudaStream_t s) {
  const int threads = norm_groups(a.d) * a.W * 32;
  return launch_pdl(norm_bwd_kernel<XT, YT, VEC, NV, PERCOL, SUMS>,
                    dim3(static_cast<unsigned>(blocks)), dim3(threads), 0, s, a);
}

template <typename XT, typename YT, int NV>
cudaError_t pick_nv(const NormArgs& a, bool vec, int blocks, cudaStream_t s) {
  const bool percol = a.gate_kind >= MOE_GATE_CHANNEL, sums = a.nsum > 0;
  if (!vec) return go<XT, YT, false, NV, true, true>(a, blocks, s);
  if (percol)
    return sums ? go<XT, YT, true, NV, true, true>(a, blocks, s)
                : go<XT, YT, true, NV, true, false>(a, blocks, s);
  return sums ? go<XT, YT, true, NV, false, true>(a, blocks, s)
              : go<XT, YT, true, NV, false, false>(a, blocks, s);
}

template <typename XT, typename YT>
cudaError_t pick(const NormArgs& a, bool vec, int blocks, cudaStream_t s) {
  switch (norm_nv(a.d)) {
    case 1: return pick_nv<XT, YT, 1>(a, vec, blocks, s);
    case 2: return pick_nv<XT, YT, 2>(a, vec, blocks, s);
    default: return pick_nv<XT, YT, 4>(a, vec, blocks, s);
  }
}

}  // namespace

cudaError_t launch_norm_bwd(const NormArgs& a, int x_type, int y_type, bool vec, int blocks,
                            float* const (&sums)[3], cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  if (blocks > 0)
    e = x_type == MOE_BF16   ? pick<bf16_t, bf16_t>(a, vec, blocks, s)
        : y_type == MOE_BF16 ? pick<float, bf16_t>(a, vec, blocks, s)
                             : pick<float, float>(a, vec, blocks, s);
  if (e != cudaSuccess || a.nsum == 0) return e;
  const int64_t n = static_cast<int64_t>(a.nsum) * a.d;
  return launch_pdl(norm_colsum_kernel, dim3(static_cast<unsigned>((n + 31) / 32)), dim3(256), 0, s,
                    static_cast<const float*>(a.part), blocks * norm_groups(a.d), a.nsum, a.d,
                    SumOuts{{sums[0], sums[1], sums[2]}});
}

}  // namespace moe
