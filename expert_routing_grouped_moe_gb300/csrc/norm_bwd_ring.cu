// Backward of the norms around a block, rows through the ring of bulk copies.
#include "norm_bwd.cuh"

namespace moe {
namespace {

template <typename XT, typename YT, bool VEC, int NV, int GATE, bool SUMS, int MAXT, int MINB>
cudaError_t go(const NormArgs& a, int blocks, cudaStream_t s) {
  auto kern = norm_bwd_kernel<XT, YT, VEC, NV, GATE, SUMS, true, MAXT, MINB>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_ring(kern, done);
  if (e != cudaSuccess) return e;
  const NormShape sh = norm_bwd_shape(a.d, true);
  return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(sh.threads()),
                    static_cast<size_t>(a.stages) * a.tile + norm_const_bytes(sh), s, a);
}

template <typename XT, typename YT, int NV, bool SUMS, int MAXT, int MINB>
cudaError_t pick_gate(const NormArgs& a, int blocks, cudaStream_t s) {
  switch (gate_class(a.gate_kind)) {
    case kGateRow: return go<XT, YT, true, NV, kGateRow, SUMS, MAXT, MINB>(a, blocks, s);
    case kGateChannel: return go<XT, YT, true, NV, kGateChannel, SUMS, MAXT, MINB>(a, blocks, s);
    default: return go<XT, YT, true, NV, kGateElement, SUMS, MAXT, MINB>(a, blocks, s);
  }
}

template <typename XT, typename YT>
cudaError_t pick(const NormArgs& a, bool vec, int blocks, cudaStream_t s) {
  const bool one = norm_bwd_shape(a.d, true).nv == 1;  // 256 threads, else up to 512
  if (!vec)
    return one ? go<XT, YT, false, 1, kGateAny, true, 256, 2>(a, blocks, s)
               : go<XT, YT, false, 2, kGateAny, true, 512, 1>(a, blocks, s);
  if (one)
    return a.nsum > 0 ? pick_gate<XT, YT, 1, true, 256, 2>(a, blocks, s)
                      : pick_gate<XT, YT, 1, false, 256, 3>(a, blocks, s);
  return a.nsum > 0 ? pick_gate<XT, YT, 2, true, 512, 1>(a, blocks, s)
                    : pick_gate<XT, YT, 2, false, 512, 1>(a, blocks, s);
}

}  // namespace

cudaError_t launch_norm_bwd_ring(const NormArgs& a, int x_type, int y_type, bool vec, int blocks,
                                 cudaStream_t s) {
  if (x_type == MOE_BF16) return pick<bf16_t, bf16_t>(a, vec, blocks, s);
  return y_type == MOE_BF16 ? pick<float, bf16_t>(a, vec, blocks, s)
                            : pick<float, float>(a, vec, blocks, s);
}

}  // namespace moe
