// Backward of the norms around a block: rows read directly, the sums over the
// blocks' partial column sums, and the choice between the two families.
#include "norm_bwd.cuh"

namespace moe {
namespace {

// The column sums: P rows of partials [nsum][d], each thread adding every 32nd
// row of one column, the 32 sums of a column then added in order; and the
// gradients they give.  Latency bounds it: ten loads a thread in flight, 304 rows
// of 4096 sums (5 MB, in the L2) in 4 us.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) norm_colsum_kernel(const NormArgs a, int P) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t n = static_cast<int64_t>(a.nsum) * a.d;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  pdl_wait();
  float t = 0.f;
  if (c < n) {
#pragma unroll 10
    for (int r = w; r < P; r += 32) t += a.part[r * n + c];
  }
  s[w][lane] = t;
  __syncthreads();
  t = s[lane][w];  // column 32 blockIdx + w
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  const int64_t cw = static_cast<int64_t>(blockIdx.x) * 32 + w;
  if (lane != 0 || cw >= n) return;
  const int q = static_cast<int>(cw / a.d), col = static_cast<int>(cw - static_cast<int64_t>(q) * a.d);
  if (q == a.sum_r) {
    a.dw_pre[col] = t;
    return;
  }
  t *= a.scale;
  float g = 1.f, dg = 0.f;
  if (a.gate_kind == MOE_GATE_CHANNEL) gate_value(static_cast<const float*>(a.gate)[col], a.sigmoid, g, dg);
  if (a.dw_post != nullptr) a.dw_post[col] = t * g;
  if (a.gate_kind == MOE_GATE_CHANNEL && a.dgate != nullptr)
    static_cast<float*>(a.dgate)[col] = t * dg * (a.w_post != nullptr ? a.w_post[col] + a.w_off : 1.f);
}

template <typename XT, typename YT, int NV>
cudaError_t go(const NormArgs& a, bool vec, int blocks, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(blocks)), threads(norm_bwd_shape(a.d, false).threads());
  return vec ? launch_pdl(norm_bwd_kernel<XT, YT, true, NV, kGateAny, true, false, 512, 1>, grid, threads, 0, s, a)
             : launch_pdl(norm_bwd_kernel<XT, YT, false, NV, kGateAny, true, false, 512, 1>, grid, threads, 0,
                          s, a);
}

template <typename XT, typename YT>
cudaError_t pick(const NormArgs& a, bool vec, int blocks, cudaStream_t s) {
  switch (norm_bwd_shape(a.d, false).nv) {
    case 1: return go<XT, YT, 1>(a, vec, blocks, s);
    case 2: return go<XT, YT, 2>(a, vec, blocks, s);
    default: return go<XT, YT, 4>(a, vec, blocks, s);
  }
}

}  // namespace

cudaError_t launch_norm_bwd_direct(const NormArgs& a, int x_type, int y_type, bool vec, int blocks,
                                   cudaStream_t s) {
  if (x_type == MOE_BF16) return pick<bf16_t, bf16_t>(a, vec, blocks, s);
  return y_type == MOE_BF16 ? pick<float, bf16_t>(a, vec, blocks, s)
                            : pick<float, float>(a, vec, blocks, s);
}

cudaError_t launch_norm_bwd(const NormArgs& args, int x_type, int y_type, bool vec, cudaStream_t s) {
  NormArgs a = args;
  const int xs = x_type == MOE_BF16 ? 2 : 4, ys = y_type == MOE_BF16 ? 2 : 4;
  const bool pre = a.w_pre != nullptr;
  NormShape sh = norm_bwd_shape(a.d, true);
  auto place = [&](int size) {
    const int bytes = sh.groups * a.d * size;
    return vec ? ring_place<true>(bytes) : ring_place<false>(bytes);
  };
  a.tile = (a.x ? place(xs) : 0) + (pre ? place(xs) + place(ys) : 0) + (a.y ? place(ys) : 0) +
           (a.gate_kind == MOE_GATE_ELEMENT ? place(ys) : 0);
  const bool barrier = pre || a.w_post || (a.gate_kind == MOE_GATE_TOKEN && a.dgate);
  const bool ring = sh.nv <= 2 && sh.W > 1 && barrier &&
                    a.T > static_cast<int64_t>(kNormRingTiles) * sh.groups;
  const bool sums = a.nsum > 0 || !vec;  // the kernels for any alignment always keep them
  int per = norm_bwd_per_sm(sh, sums);
  a.stages = ring ? ring_stages(a.tile, &per, norm_const_bytes(sh), kBwdFlight) : 0;
  if (a.stages == 0) sh = norm_bwd_shape(a.d, false);
  a.W = sh.W;
  const int blocks = norm_bwd_blocks(sh, a.T, sums);
  const cudaError_t e = a.stages > 0 ? launch_norm_bwd_ring(a, x_type, y_type, vec, blocks, s)
                                     : launch_norm_bwd_direct(a, x_type, y_type, vec, blocks, s);
  if (e != cudaSuccess || a.nsum == 0) return e;
  const int64_t n = static_cast<int64_t>(a.nsum) * a.d;
  return launch_pdl(norm_colsum_kernel, dim3(static_cast<unsigned>((n + 31) / 32)), dim3(kSumThreads),
                    0, s, a, blocks * sh.groups);
}

}  // namespace moe
