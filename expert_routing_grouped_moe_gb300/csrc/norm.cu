// C ABI of the norms around a block: argument checks and launches.
#include <cmath>

#include "norm.cuh"

namespace moe {
namespace {

int bad(const char* msg) { return record_error(MOE_ERR_INVALID_ARG, msg); }

// Type-dependent alignment every pointer must have, and 16 bytes for the
// vector path: vec is cleared where a pointer or d does not allow it.
bool aligned(const void* p, size_t size, bool& vec) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(p);
  if (u & 15u) vec = false;
  return (u & (size - 1)) == 0;
}

int check_desc(const moe_norm_desc* q) {
  if (q == nullptr) return bad("desc is NULL");
  if (q->T < 0 || q->d <= 0) return bad("T must not be negative, d must be positive");
  if (q->d > kNormMaxD) return record_error(MOE_ERR_UNSUPPORTED, "d > MOE_NORM_MAX_D");
  if ((q->x_type != MOE_F32 && q->x_type != MOE_BF16) ||
      (q->y_type != MOE_F32 && q->y_type != MOE_BF16))
    return bad("x_type and y_type must be MOE_F32 or MOE_BF16");
  if (q->x_type == MOE_BF16 && q->y_type == MOE_F32)
    return record_error(MOE_ERR_UNSUPPORTED, "a bf16 residual stream needs a bf16 block output");
  if (q->gate < MOE_GATE_NONE || q->gate > MOE_GATE_ELEMENT) return bad("bad gate kind");
  if (q->gate_sigmoid != 0 && q->gate_sigmoid != 1) return bad("gate_sigmoid must be 0 or 1");
  if (!(q->eps > 0.f) || !std::isfinite(q->eps)) return bad("eps must be positive");
  if (!std::isfinite(q->scale) || !std::isfinite(q->w_offset))
    return bad("scale and w_offset must be finite");
  return MOE_OK;
}

size_t size_of(int type) { return type == MOE_BF16 ? 2 : 4; }

// wide: cleared where p does not allow 16-byte vectors (values read one by one,
// such as [T] vectors, have a flag of their own that nothing reads)
#define NORM_PTR(p, size, wide)                                   \
  do {                                                            \
    if ((p) == nullptr) return bad(#p " is NULL");                \
    if (!aligned(p, size, wide)) return bad(#p " is misaligned"); \
  } while (0)

// Self-test of the ring's failure path: one block of two warps passes its rows
// through the norms' own ring.  Warp `late` (0: the one that fills the ring, at the
// third tile; 1: the other, at the last; -1: none) waits there for a barrier that
// nothing arrives on, and gives up after the limit.  *tiles: how many tiles were
// filled, or -1 where one of them was still in flight at the end.
constexpr int kSelfRows = 8, kSelfStages = 2, kSelfD = 64;
__device__ __align__(16) float g_selftest_rows[kSelfRows * kSelfD];
__global__ void __launch_bounds__(64) ring_selftest_kernel(int late, uint64_t limit_ns, int32_t* tiles,
                                                           int* status) {
  __shared__ __align__(128) uint8_t s_tiles[kSelfStages * kSelfD * 4];
  __shared__ RingState s_ring;
  __shared__ uint64_t s_never;
  const RingSrc src[kRingSrcs] = {{g_selftest_rows, 4}, {nullptr, 0}, {nullptr, 0}, {nullptr, 0}, {nullptr, 0}};
  const int place = kSelfD * 4;
  int filled = 0;
  auto fill = [&](int stage, int64_t row) {
    ring_fill<true>(src, s_tiles + stage * place, &s_ring.full[stage], row, kSelfRows, 1, kSelfD);
    ++filled;
  };
  if (threadIdx.x == 0) {
    mbar_init(&s_never, 1);
    ring_init(s_ring, kSelfStages);
  }
  __syncthreads();
  if (threadIdx.x == 0)
    for (int q = 0; q < kSelfStages; ++q) fill(q, q);
  int stage = 0, phase = 0, before = 0;
  bool filling = true;
  for (int64_t base = 0; base < kSelfRows; ++base) {
    const bool miss = base == (late == 0 ? 2 : kSelfRows - 1) && static_cast<int>(threadIdx.x >> 5) == late;
    filling &= ring_wait(s_ring, miss ? &s_never : &s_ring.full[stage], stage, miss ? 0 : phase, base, status, limit_ns);
    __syncthreads();
    if (threadIdx.x == 0 && filling && base >= 1 && base + kSelfStages - 1 < kSelfRows)
      fill(before, base + kSelfStages - 1);
    before = stage;
    if (++stage == kSelfStages) { stage = 0; phase ^= 1; }
  }
  ring_drain(s_ring, kSelfStages, 1, kSelfRows);
  if (threadIdx.x == 0) {
    for (int t = filled - kSelfStages; t < filled; ++t)  // each place's last tile has landed
      if (!mbar_try_wait(&s_ring.full[t % kSelfStages], (t / kSelfStages) & 1)) filled = -1;
    *tiles = filled;
  }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_block_norm_fwd(const moe_norm_desc* desc, const void* x, const void* y, const void* gate,
                       const float* w_post, const float* w_pre, void* r, void* n, float* rstd_y,
                       float* rstd_r, moe_stream_t stream) {
  NvtxScope nvtx("moe_block_norm_fwd");
  int rc = check_desc(desc);
  if (rc) return rc;
  if (desc->T == 0) return record_error(MOE_OK, "");
  const size_t xs = size_of(desc->x_type), ys = size_of(desc->y_type);
  bool vec = desc->d % 8 == 0, per_row = true;
  if (x == nullptr && y == nullptr) return bad("x and y are both NULL");
  if (y == nullptr && (r != nullptr || w_post != nullptr || desc->gate != MOE_GATE_NONE))
    return bad("r, w_post and a gate go with y");
  if (y == nullptr && w_pre == nullptr) return bad("nothing to compute: no y and no w_pre");
  if ((w_pre == nullptr) != (n == nullptr)) return bad("w_pre and n go together");
  if ((gate == nullptr) != (desc->gate == MOE_GATE_NONE)) return bad("gate and its kind go together");
  if (x) NORM_PTR(x, xs, vec);
  if (y) { NORM_PTR(y, ys, vec); NORM_PTR(r, xs, vec); }
  if (desc->gate == MOE_GATE_TOKEN) NORM_PTR(gate, 4, per_row);
  else if (gate) NORM_PTR(gate, (desc->gate == MOE_GATE_ELEMENT ? ys : 4), vec);
  if (w_post) { NORM_PTR(w_post, 4, vec); NORM_PTR(rstd_y, 4, per_row); }
  if (w_pre) { NORM_PTR(w_pre, 4, vec); NORM_PTR(n, ys, vec); NORM_PTR(rstd_r, 4, per_row); }
  NormArgs a = {};
  a.x = x; a.y = y; a.gate = gate; a.w_post = w_post; a.w_pre = w_pre;
  a.r = r; a.n = n; a.rstd_y = rstd_y; a.rstd_r = rstd_r;
  a.T = desc->T; a.d = desc->d;
  a.gate_kind = desc->gate; a.sigmoid = desc->gate_sigmoid;
  a.scale = desc->scale; a.eps = desc->eps; a.w_off = desc->w_offset;
  rc = device_status_word(&a.status);
  if (rc != MOE_OK) return rc;
  ProbeScope probe("block_norm_fwd", stream);
  const cudaError_t e = launch_norm_fwd(a, desc->x_type, desc->y_type, vec, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

size_t moe_block_norm_workspace_size(int32_t T, int32_t d) {
  if (T < 0 || d <= 0 || d > kNormMaxD) return 0;
  size_t rows = 0;  // the larger of the two ways to read rows
  for (const bool ring : {false, true}) {
    const NormShape sh = norm_bwd_shape(d, ring);
    const size_t r = static_cast<size_t>(norm_bwd_blocks(sh, T, true)) * sh.groups;
    rows = r > rows ? r : rows;
  }
  return rows * 2 * static_cast<size_t>(d) * 4;
}

int moe_block_norm_bwd(const moe_norm_desc* desc, const void* dr, const void* dn, const void* r,
                       const void* y, const void* gate, const float* w_post, const float* w_pre,
                       const float* rstd_y, const float* rstd_r, void* dx, void* dy, void* dgate,
                       float* dw_post, float* dw_pre, void* ws, size_t ws_bytes,
                       moe_stream_t stream) {
  NvtxScope nvtx("moe_block_norm_bwd");
  int rc = check_desc(desc);
  if (rc) return rc;
  // sums over the tokens, the only outputs that T = 0 has
  NormArgs a = {};
  const bool sum_gate = dgate != nullptr && desc->gate == MOE_GATE_CHANNEL;
  a.sum_y = dw_post != nullptr || sum_gate ? a.nsum++ : -1;
  a.sum_r = dw_pre != nullptr ? a.nsum++ : -1;
  for (const void* p : {static_cast<const void*>(dw_post), static_cast<const void*>(dw_pre),
                        static_cast<const void*>(sum_gate ? dgate : nullptr)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return bad("a sum over the tokens is misaligned");
  if ((dgate && !gate) || (dw_post && !w_post) || (dw_pre && !w_pre))
    return bad("the gradient of an input that is not there");
  // without tokens, a gate for each token or element has nothing to point to
  const bool no_gate_values = desc->T == 0 && (desc->gate == MOE_GATE_TOKEN || desc->gate == MOE_GATE_ELEMENT);
  if (!no_gate_values && (gate == nullptr) != (desc->gate == MOE_GATE_NONE))
    return bad("gate and its kind go together");
  for (const void* p : {desc->gate == MOE_GATE_CHANNEL ? gate : nullptr, static_cast<const void*>(w_post)})
    if (reinterpret_cast<uintptr_t>(p) & 3u) return bad("a vector of d values is misaligned");
  a.dw_post = dw_post; a.dw_pre = dw_pre; a.gate = gate; a.dgate = dgate;
  a.w_post = w_post; a.w_pre = w_pre;
  a.gate_kind = desc->gate; a.sigmoid = desc->gate_sigmoid;
  a.scale = desc->scale; a.eps = desc->eps; a.w_off = desc->w_offset;
  a.T = desc->T; a.d = desc->d;
  if (desc->T == 0) {  // zeros, whatever the gate and the weights hold
    for (void* p : {static_cast<void*>(dw_post), static_cast<void*>(dw_pre), sum_gate ? dgate : nullptr}) {
      if (p == nullptr) continue;
      const cudaError_t e = cudaMemsetAsync(p, 0, static_cast<size_t>(desc->d) * 4, stream);
      if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
    }
    return record_error(MOE_OK, "");
  }
  const size_t xs = size_of(desc->x_type), ys = size_of(desc->y_type);
  bool vec = desc->d % 8 == 0, per_row = true;
  if (dr == nullptr && dn == nullptr) return bad("dr and dn are both NULL");
  if ((w_pre == nullptr) != (dn == nullptr)) return bad("w_pre and dn go together");
  if (y == nullptr && (w_post != nullptr || dy != nullptr || desc->gate != MOE_GATE_NONE))
    return bad("w_post, dy and a gate go with y");
  if (dx == nullptr && dy == nullptr && dgate == nullptr && dw_post == nullptr && dw_pre == nullptr)
    return bad("nothing to compute");
  if (dr) NORM_PTR(dr, xs, vec);
  if (dn) {
    NORM_PTR(dn, ys, vec); NORM_PTR(r, xs, vec); NORM_PTR(w_pre, 4, vec);
    NORM_PTR(rstd_r, 4, per_row);
  }
  if (y) NORM_PTR(y, ys, vec);
  if (w_post) { NORM_PTR(w_post, 4, vec); NORM_PTR(rstd_y, 4, per_row); }
  if (desc->gate == MOE_GATE_TOKEN) NORM_PTR(gate, 4, per_row);
  else if (gate) NORM_PTR(gate, (desc->gate == MOE_GATE_ELEMENT ? ys : 4), vec);
  if (dx) NORM_PTR(dx, xs, vec);
  if (dy) NORM_PTR(dy, ys, vec);
  if (dgate && desc->gate == MOE_GATE_TOKEN) NORM_PTR(dgate, 4, per_row);
  if (dgate && desc->gate == MOE_GATE_ELEMENT) NORM_PTR(dgate, ys, vec);
  if (a.nsum > 0) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 15u)) return bad("ws NULL or misaligned");
    if (ws_bytes < moe_block_norm_workspace_size(desc->T, desc->d))
      return record_error(MOE_ERR_WORKSPACE, "norm workspace too small");
  }
  a.x = dr; a.y = y;
  a.r = const_cast<void*>(r); a.n = const_cast<void*>(dn);
  a.rstd_y = const_cast<float*>(rstd_y); a.rstd_r = const_cast<float*>(rstd_r);
  a.dx = dx; a.dy = dy;
  a.part = static_cast<float*>(ws);
  rc = device_status_word(&a.status);
  if (rc != MOE_OK) return rc;
  ProbeScope probe("block_norm_bwd", stream);
  const cudaError_t e =
      launch_norm_bwd(a, desc->x_type, desc->y_type, vec, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

int moe_selftest_ring_timeout(uint32_t timeout_us, int32_t late, int32_t* tiles, moe_stream_t stream) {
  if (timeout_us == 0 || timeout_us > 2000000u) return bad("timeout_us must be in (0, 2000000]");
  if (late < -1 || late > 1) return bad("late must be -1, 0 or 1");
  if (tiles == nullptr || (reinterpret_cast<uintptr_t>(tiles) & 3u)) return bad("tiles NULL or misaligned");
  int* status = nullptr;
  const int rc = device_status_word(&status);
  if (rc != MOE_OK) return rc;
  ring_selftest_kernel<<<1, 64, 0, stream>>>(late, static_cast<uint64_t>(timeout_us) * 1000u, tiles, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
