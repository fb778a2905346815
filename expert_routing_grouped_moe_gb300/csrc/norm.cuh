// Kernels of the norms around a block, forward and backward (norm_fwd.cu,
// norm_bwd.cu): what the two share.
#pragma once

#include <atomic>
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
  float *dw_post, *dw_pre;
  int sum_y, sum_r;   // index of each column sum in part, -1: not wanted
  int nsum;
  int64_t T;
  int d, W;           // columns; warps that share a row
  int gate_kind, sigmoid;
  float scale, eps, w_off;
  int stages, tile;   // ring: tiles held and bytes of one; 0: rows are read directly
  int* status;
};

// The vectors [d] that a kernel applies to every row are kept in registers while
// a thread has at most two shares of a row, else read again for each row.
template <int NV>
struct RowConst {
  f2 f[NV <= 2 ? NV : 1][4];
};

// A row's shares: NV of 8 values for each thread of W <= 16 warps, 32 W NV 8 >= d;
// as many groups of W warps, a row each, as fill 8 warps.
constexpr int kNormMaxWarps = 16;
constexpr int kNormMaxD = kNormMaxWarps * 32 * 8 * 4;
struct NormShape {
  int nv, W, groups;
  int threads() const { return 32 * W * groups; }
};
inline NormShape norm_shape(int d, int nv) {
  NormShape s;
  s.nv = nv;
  s.W = (d + 256 * nv - 1) / (256 * nv);
  s.groups = s.W >= 8 ? 1 : 8 / s.W;
  return s;
}
// Forward: two shares for each thread beyond 1024 columns (fewer warps to wait for
// one another; 4096x2048 12.9 us, with one share 16.4).
inline NormShape norm_fwd_shape(int d) { return norm_shape(d, d <= 1024 ? 1 : d <= 8192 ? 2 : 4); }
// Backward, rows read directly: one share for each thread while that takes 16
// warps at most.  Through the ring: one up to 2048 columns, where two save
// nothing (16384x2048 83 us and 85), two above (frozen weights, 16384x2880: 96 us,
// with one 110; 4096 columns: 142, with one share no second block fits).
inline NormShape norm_bwd_shape(int d, bool ring) {
  return norm_shape(d, d <= (ring ? 2048 : 4096) ? 1 : d <= 8192 ? 2 : 4);
}

// Sums v[0..K) (K = 1 or 3) over the W <= 16 warps of this thread's row group;
// all threads of the block call it.  buf: 16 warps x 4 values, one of two
// arrays that the caller alternates, so one barrier per call is enough: a warp
// writes an array again only after the barrier of the call in between, which
// every reader has passed.
// Three sums: the first two exchanges halve what a lane carries (lanes 0-7 end
// with v[0], 8-15 with v[1], 16-23 with v[2]): 6 shuffles instead of 15.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*buf)[4], int W, int warp, int first) {
  constexpr unsigned kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  if (K == 1) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[0] += __shfl_xor_sync(kAll, v[0], o);
    if (W == 1) return;
    if (lane == 0) buf[warp][0] = v[0];
    __syncthreads();
    float t = (lane & 15) < W ? buf[first + (lane & 15)][0] : 0.f;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(kAll, t, o);
    v[0] = t;
  } else {
    const bool up = lane & 16, right = lane & 8;
    const float s0 = __shfl_xor_sync(kAll, up ? v[0] : v[2], 16);
    const float s1 = __shfl_xor_sync(kAll, up ? v[1] : 0.f, 16);
    const float x = (up ? v[2] : v[0]) + s0, y = (up ? 0.f : v[1]) + s1;  // up: y unused
    float t = (right ? y : x) + __shfl_xor_sync(kAll, right ? x : y, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) t += __shfl_xor_sync(kAll, t, o);
    if (W == 1) {
      v[0] = __shfl_sync(kAll, t, 0);
      v[1] = __shfl_sync(kAll, t, 8);
      v[2] = __shfl_sync(kAll, t, 16);
      return;
    }
    if ((lane & 7) == 0) buf[warp][lane >> 3] = t;
    __syncthreads();
    const int q = lane >> 2;
    t = q < W ? buf[first + q][lane & 3] : 0.f;
    if (q + 8 < W) t += buf[first + q + 8][lane & 3];
#pragma unroll
    for (int o = 16; o >= 4; o >>= 1) t += __shfl_xor_sync(kAll, t, o);
    v[0] = __shfl_sync(kAll, t, 0);
    v[1] = __shfl_sync(kAll, t, 1);
    v[2] = __shfl_sync(kAll, t, 2);
  }
}

// a(gate) and its derivative; sigmoid from e^-|g|, so neither a nor 1 - a cancels.
__device__ __forceinline__ void gate_value(float g, int sigmoid, float& a, float& da) {
  if (sigmoid) {
    const float e = expf(-fabsf(g));
    const float big = __fdividef(1.f, 1.f + e), small = e * big;
    a = g >= 0.f ? big : small;
    da = big * small;
    if (g != g) a = da = g;
  } else {
    a = g;
    da = 1.f;
  }
}

__device__ __forceinline__ f2 gate_pair(f2 g, int sigmoid) {
  if (!sigmoid) return g;
  const float2 x = unpk(g);
  float a, b, unused;
  gate_value(x.x, 1, a, unused);
  gate_value(x.y, 1, b, unused);
  return pk(a, b);
}

// How a kernel is told the gate's kind: fixed when it is compiled, or GATE_ANY.
constexpr int kGateRow = 0, kGateChannel = 1, kGateElement = 2, kGateAny = 3;
template <int GATE>
__device__ __forceinline__ bool gate_is(int kind, int want) {
  if (GATE == kGateRow) return false;
  if (GATE == kGateChannel) return want == MOE_GATE_CHANNEL;
  if (GATE == kGateElement) return want == MOE_GATE_ELEMENT;
  return kind == want;
}
inline int gate_class(int kind) {
  return kind == MOE_GATE_CHANNEL ? kGateChannel : kind == MOE_GATE_ELEMENT ? kGateElement : kGateRow;
}

// ---- rows staged through shared memory ---------------------------------------
// A tile is the rows of a block's groups, consecutive in memory: one bulk copy
// for each input.  A ring of `stages` tiles is filled ahead by one thread; a
// tile's place is filled again after the first block-wide barrier of the next
// tile, which every thread reaches after its last read of this one.
// Bulk copies move 16-byte words.  Where rows do not begin and end on them
// (VEC false) the words around a tile's first and last value come along, and
// its values lie as far into their place as they lie into the first word; what
// would reach past either end of the tensor is copied value by value instead.
struct RingSrc {
  const void* p;   // [T,d] input, NULL: none
  int esize;       // bytes of an element
};
constexpr int kRingSrcs = 5, kRingMaxStages = 4;
constexpr int kRingBytes = 208 * 1024;  // of an SM's shared memory
// A ring's barriers, and where the thread that fills it (thread 0) gave up waiting.
struct RingState {
  uint64_t full[kRingMaxStages];
  int64_t lost_base;  // first row of that tile
  int abort, lost_stage, lost_phase;
};
__device__ __forceinline__ void ring_init(RingState& r, int stages) {  // thread 0
  r.abort = 0;
  r.lost_base = -1;
  for (int q = 0; q < stages; ++q) mbar_init(&r.full[q], 1);
  fence_mbar_init();
}
// Waits for a tile.  Every thread waits by its own clock, so any of them may be the
// only one that gives up (false), and each that does raises the status word.  Thread 0
// fills no more from there on: a place it has not seen filled may still be written.
__device__ __forceinline__ bool ring_wait(RingState& r, uint64_t* bar, int stage, int phase, int64_t base,
                                          int* status, uint64_t limit_ns) {
  if (mbar_wait(bar, phase, &r.abort, limit_ns)) return true;
  atomicCAS(status, 0, kErrTimeout);
  if (threadIdx.x == 0 && r.lost_base < 0) {
    r.lost_base = base;
    r.lost_stage = stage;
    r.lost_phase = phase;
  }
  return false;
}
// Before thread 0 leaves the kernel: the copies still in flight where it gave up,
// once more with a limit.  Those are the tiles from that one on that were filled:
// all of the first `stages`, and one fewer once tiles follow them.
__device__ __forceinline__ void ring_drain(RingState& r, int stages, int64_t step, int64_t T) {
  if (threadIdx.x != 0 || r.lost_base < 0) return;
  int never = 0, stage = r.lost_stage, phase = r.lost_phase;
  const int filled = stages - (r.lost_base >= step ? 1 : 0);
  for (int q = 0; q < filled && r.lost_base + q * step < T; ++q) {
    mbar_wait(&r.full[stage], phase, &never, 1000000000ull);
    if (++stage == stages) { stage = 0; phase ^= 1; }
  }
}

// Bytes of a tile's place for `bytes` of rows.
template <bool VEC>
__host__ __device__ __forceinline__ int ring_place(int bytes) {
  return VEC ? bytes : (bytes + 30) & ~15;
}
// The first row of the tile at row `base` within its place.
template <bool VEC, typename T>
__device__ __forceinline__ const T* ring_row(const uint8_t* place, const T* src, int64_t base, int d) {
  return reinterpret_cast<const T*>(
      place + (VEC ? 0 : static_cast<int>(reinterpret_cast<uintptr_t>(src + base * d) & 15u)));
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// The words of one input's tile: [from, to) of memory, the rest of [begin, end)
// outside them at most 15 bytes on either side.
struct RingSpan {
  uintptr_t begin, end, from, to;
};
template <bool VEC>
__device__ __forceinline__ RingSpan ring_span(const RingSrc& q, int64_t base, int rows, int64_t T, int d) {
  RingSpan s;
  s.begin = reinterpret_cast<uintptr_t>(q.p) + static_cast<uintptr_t>(base * d * q.esize);
  s.end = s.begin + static_cast<uintptr_t>(rows) * d * q.esize;
  s.from = s.begin;
  s.to = s.end;
  if (!VEC) {
    s.from = base == 0 ? (s.begin + 15) & ~uintptr_t(15) : s.begin & ~uintptr_t(15);
    s.to = base + rows == T ? s.end & ~uintptr_t(15) : (s.end + 15) & ~uintptr_t(15);
    if (s.to < s.from) s.to = s.from = s.begin & ~uintptr_t(15);  // within one word: value by value
  }
  return s;
}
// The tile of rows [base, base + groups) into `stage`; inputs one after the other.
template <bool VEC>
__device__ __forceinline__ void ring_fill(const RingSrc (&src)[kRingSrcs], uint8_t* stage,
                                          uint64_t* bar, int64_t base, int64_t T, int groups, int d) {
  const int64_t left = T - base;
  const int rows = left < groups ? static_cast<int>(left) : groups;
  uint32_t total = 0;
  int at = 0;
#pragma unroll
  for (int i = 0; i < kRingSrcs; ++i) {
    if (src[i].p == nullptr) continue;
    const RingSpan s = ring_span<VEC>(src[i], base, rows, T, d);
    total += static_cast<uint32_t>(s.to - s.from);
    if (!VEC) {  // before the barrier's arrival, which makes them visible
      const int es = src[i].esize;
      const uintptr_t word = s.begin & ~uintptr_t(15);
      auto one_by_one = [&](uintptr_t p, uintptr_t end) {
        for (; p < end; p += es) {
          uint8_t* to = stage + at + static_cast<int>(p - word);
          if (es == 2) *reinterpret_cast<uint16_t*>(to) = *reinterpret_cast<const uint16_t*>(p);
          else *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(p);
        }
      };
      one_by_one(s.begin, s.from < s.end ? s.from : s.end);
      one_by_one(s.to > s.begin ? s.to : s.begin, s.end);
      at += ring_place<VEC>(groups * d * es);
    }
  }
  // values stored by this thread come before the copies that fill the place again
  if (!VEC && (base == 0 || base + rows == T)) fence_proxy_async_smem();
  mbar_expect_tx(bar, total);
  at = 0;
#pragma unroll
  for (int i = 0; i < kRingSrcs; ++i) {
    if (src[i].p == nullptr) continue;
    const RingSpan s = ring_span<VEC>(src[i], base, rows, T, d);
    if (VEC || s.to > s.from)
      bulk_load(stage + at + (VEC ? 0 : static_cast<int>(s.from - (s.begin & ~uintptr_t(15)))),
                reinterpret_cast<const void*>(s.from), static_cast<uint32_t>(s.to - s.from), bar);
    at += ring_place<VEC>(groups * d * src[i].esize);
  }
}

// Rows of two and more shares read directly: the words of row `row` of each input
// that lie in it whole, into the L2 while the row before is worked on.  For up to
// 160 KB of inputs a row (backward of 4096x12000 in bf16, 96 KB: 374 us, without
// 447; of 4096x8192 in fp32 with an element gate, 160 KB: 285 and 295; of
// 4096x12000 so, 240 KB: 762 and 637).
constexpr int kPrefetchBytes = 160 * 1024;
__device__ __forceinline__ void prefetch_row(const RingSrc (&src)[kRingSrcs], int64_t row, int d) {
#pragma unroll
  for (int i = 0; i < kRingSrcs; ++i) {
    if (src[i].p == nullptr) continue;
    const uintptr_t at = reinterpret_cast<uintptr_t>(src[i].p) + static_cast<uintptr_t>(row * d * src[i].esize);
    const uintptr_t from = (at + 15) & ~uintptr_t(15),
                    to = (at + static_cast<uintptr_t>(d) * src[i].esize) & ~uintptr_t(15);
    if (to > from)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from),
                   "r"(static_cast<uint32_t>(to - from)) : "memory");
  }
}

// Lets a kernel use the ring's shared memory, once on each device.
template <typename Kernel>
cudaError_t allow_ring(Kernel kern, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Stages of a ring of `tile` bytes each for up to *per blocks on an SM (each with
// `extra` bytes besides): as many, from 2 to 4, as keep at most `flight` bytes on
// their way to an SM; fewer blocks where two stages each do not fit, 0 when they
// do not fit one.  The forward does best with about 100 KB in flight (16384x2880
// 62 us; 67.6 with 138 KB, 85 with 46), the backward, which computes longer on a
// tile, with all that fits (frozen weights, 16384x2048: 70 us, 83 with 98 KB).
constexpr int kFwdFlight = 104 * 1024, kBwdFlight = kRingBytes;
inline int ring_stages(size_t tile, int* per, size_t extra, int64_t flight) {
  for (; *per > 0; --*per) {
    const int64_t room = kRingBytes / *per - static_cast<int64_t>(extra), t = static_cast<int64_t>(tile);
    if (room < 2 * t) continue;
    const int64_t fit = room / t, want = flight / (*per * t), n = want < fit ? want : fit;
    return n < 2 ? 2 : n < kRingMaxStages ? static_cast<int>(n) : kRingMaxStages;
  }
  return 0;
}
// The backward's two vectors of per-column factors.
inline size_t norm_const_bytes(const NormShape& s) { return static_cast<size_t>(s.threads()) * s.nv * 64; }
// Fewer tiles than this are read directly (a block would have one or two).
constexpr int kNormRingTiles = 2 * kSMs;

// Blocks of the backward: what the SMs' registers hold, at 128 a thread where
// they keep column sums or two shares, at 80 otherwise.  Those that keep column
// sums write a row of partial sums for each of their groups.
inline int norm_bwd_per_sm(const NormShape& s, bool sums) {
  return !sums && s.nv == 1 && s.threads() <= 256 ? 3 : s.threads() <= 256 ? 2 : 1;
}
inline int norm_bwd_blocks(const NormShape& s, int64_t T, bool sums) {
  const int64_t need = (T + s.groups - 1) / s.groups, most = norm_bwd_per_sm(s, sums) * kSMs;
  return static_cast<int>(need < most ? need : most);
}

cudaError_t launch_norm_fwd(const NormArgs& a, int x_type, int y_type, bool vec, cudaStream_t s);
cudaError_t launch_norm_bwd(const NormArgs& a, int x_type, int y_type, bool vec, cudaStream_t s);

}  // namespace moe
