// Rows of a table for token ids, and the table's gradient.
//   out[t] = scale table[ids[t]]
//   dtable[v] = scale sum_{t: ids[t] = v} dout[t]     (dense, or added)
// Forward: a copy of rows, bound by memory.
//
// Gradient.  The tokens are sorted by id: a stable radix sort, least digit first,
// of up to 9 bits a pass, so two passes for a table of up to 2^18 rows; up to
// 65536 tokens in one launch of one cluster, which keeps them in its shared
// memory between passes, while a second kernel writes the zeros.  Sorted
// tokens are cut into chunks of equal length, and a group of threads walks one
// chunk with 8 columns a thread: it adds up rows while the id stays the same and
// writes a run that lies in its chunk straight to the table.  A run that reaches
// over chunk borders leaves its parts in the workspace, [chunk][first, last], and
// a second kernel adds them in order.  So the work is even whatever the ids'
// frequencies, nothing is atomic, and the order of every sum depends on the ids and the
// width alone.  What bounds it: T d reads of gradient rows and, dense, V d writes of
// which most are zeros.  4096 x 2048 into 151936 rows, dense: 179 us (186 at a copy's
// rate; the zeros alone 162, all else runs beside them), 32768 x 2048: 225.  Added to a
// table instead, 4096 x 2048: 34 us, three launches that wait for one another.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

// Lets the next kernel of the stream start while this one runs.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ---- forward -----------------------------------------------------------------
// A warp moves up to 256 SH columns of a row, SH shares of 8 a lane: four where that
// leaves every SM its 64 warps, else two.
constexpr int kFwdThreads = 256, kFwdWarps = kFwdThreads / 32;

__device__ __forceinline__ void put_share(bf16_t* row, int v, const f2 (&f)[4], bool) {
  Raw8<bf16_t> r;
  narrow(f, r);
  *(reinterpret_cast<uint4*>(row) + v) = r.v;
}
// wide: rows are 32-byte aligned, and a share is one access (see store8_wide).
__device__ __forceinline__ void put_share(float* row, int v, const f2 (&f)[4], bool wide) {
  Raw8<float> r;
  narrow(f, r);
  if (wide) {
    store8_wide(row + 8 * v, r);
  } else {
    *(reinterpret_cast<float4*>(row) + 2 * v) = r.a;
    *(reinterpret_cast<float4*>(row) + 2 * v + 1) = r.b;
  }
}

template <typename T, typename O, bool VEC, int SH>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const void* __restrict__ ids, int id64,
                                                               const T* __restrict__ table, int64_t T_, int V,
                                                               int d, float scale, O* __restrict__ out, bool wide,
                                                               int* status) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const unsigned segs = (d + 256 * SH - 1) / (256 * SH);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kFwdWarps + (threadIdx.x >> 5);
  const int64_t t = (unit >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(unit) / segs) : unit / segs;
  if (t >= T_) return;
  const int v0 = static_cast<int>(unit - t * segs) * 32 * SH + lane;
  const int64_t id = id64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
  const bool ok = id >= 0 && id < V;
  if (!ok && lane == 0) atomicCAS(status, 0, kErrBadIds);
  const T* from = table + (ok ? id : 0) * static_cast<int64_t>(d);
  O* to = out + t * d;
  Raw8<T> raw[SH];
#pragma unroll
  for (int i = 0; i < SH; ++i) load8<VEC>(from, v0 + 32 * i, d, raw[i]);
  const f2 s = pk(scale);
#pragma unroll
  for (int i = 0; i < SH; ++i) {
    f2 f[4];
    widen(raw[i], f);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = ok ? mul2(f[e], s) : pk(0.f);
    if (!VEC) put8<O, VEC>(to, v0 + 32 * i, d, f);
    else if (8 * (v0 + 32 * i) < d) put_share(to, v0 + 32 * i, f, wide);
  }
}

// ---- sort --------------------------------------------------------------------
constexpr int kMaxDigit = 9, kMaxBins = 1 << kMaxDigit;
constexpr int kSortThreads = 256, kSortWarps = kSortThreads / 32, kSortRounds = 16;
constexpr int kSortChunk = kSortThreads * kSortRounds;  // tokens of a block

// The digits of a table of V rows: ids 0 .. V - 1, and V for tokens that add nothing.
struct Digits {
  int passes, bits;
};
__host__ __device__ inline Digits digits(int V) {
  int n = 1;
  while (n < 31 && (V >> n) != 0) ++n;
  const int passes = (n + kMaxDigit - 1) / kMaxDigit;
  return {passes, (n + passes - 1) / passes};
}

// The id a token is sorted by.
__device__ __forceinline__ uint32_t key_of(const void* ids, int id64, int64_t t, int V, int64_t pad, int* status) {
  const int64_t id = id64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
  if (id == pad && pad >= 0) return static_cast<uint32_t>(V);
  if (id >= 0 && id < V) return static_cast<uint32_t>(id);
  if (status != nullptr) atomicCAS(status, 0, kErrBadIds);
  return static_cast<uint32_t>(V);
}

// Where a pass reads its keys and tokens: the ids themselves, or the pass before.
struct Source {
  const void* ids;   // nullptr: keys and tokens
  const uint32_t *keys, *tokens;
  int id64, V;
  int64_t pad;
};
__device__ __forceinline__ uint32_t source_key(const Source& s, int64_t i, int* status) {
  return s.ids != nullptr ? key_of(s.ids, s.id64, i, s.V, s.pad, status) : s.keys[i];
}

// The lanes of `live` with this lane's digit, by a vote on each of its bits (matching the
// digits by one instruction takes longer where most of them differ: the sort of 65536
// tokens 33 us against 29).
__device__ __forceinline__ unsigned lanes_with(uint32_t digit, int bits, unsigned live) {
  unsigned same = live;
#pragma unroll
  for (int b = 0; b < kMaxDigit; ++b) {
    if (b >= bits) break;
    const bool one = (digit >> b) & 1u;
    const unsigned vote = __ballot_sync(0xffffffffu, one);
    same &= one ? vote : ~vote;
  }
  return same;
}

// counts[bin][chunk] of this pass's digit.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const Source src, int64_t n, int shift, int bins,
                                                                 int chunks, uint32_t* __restrict__ counts,
                                                                 int* status) {
  __shared__ uint32_t s_count[kMaxBins];
  for (int b = threadIdx.x; b < bins; b += kSortThreads) s_count[b] = 0;
  pdl_wait();
  __syncthreads();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortChunk;
#pragma unroll 4
  for (int i = 0; i < kSortRounds; ++i) {
    const int64_t t = base + i * kSortThreads + threadIdx.x;
    if (t < n) atomicAdd(&s_count[(source_key(src, t, status) >> shift) & (bins - 1)], 1u);
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads)
    counts[static_cast<int64_t>(b) * chunks + blockIdx.x] = s_count[b];
}

// Exclusive sums of n counts in place, by one block.
constexpr int kScanThreads = 1024, kScanEach = 8;
__global__ void __launch_bounds__(kScanThreads) sort_scan_kernel(uint32_t* __restrict__ counts, int64_t n) {
  __shared__ uint32_t s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t before = 0;
  pdl_wait();
  for (int64_t base = 0; base < n; base += kScanThreads * kScanEach) {
    const int64_t at = base + static_cast<int64_t>(threadIdx.x) * kScanEach;
    uint32_t v[kScanEach], sum = 0;
#pragma unroll
    for (int e = 0; e < kScanEach; ++e) {
      v[e] = at + e < n ? counts[at + e] : 0u;
      sum += v[e];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t q = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += q;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
      uint32_t w = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t q = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += q;
      }
      s_warp[lane] = w;
    }
    __syncthreads();
    uint32_t run = before + (warp > 0 ? s_warp[warp - 1] : 0u) + incl - sum;
#pragma unroll
    for (int e = 0; e < kScanEach; ++e) {
      if (at + e < n) counts[at + e] = run;
      run += v[e];
    }
    before += s_warp[31];
    __syncthreads();
  }
}

// Tokens to their places.  Each warp takes a run of its block's tokens; lanes with the
// same digit find each other, so that a token's rank in its bin is what the warps
// before, the rounds before and the lanes before hold.
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const Source src, int64_t n, int shift, int bits,
                                                                 int chunks, const uint32_t* __restrict__ starts,
                                                                 uint32_t* __restrict__ keys,
                                                                 uint32_t* __restrict__ tokens) {
  __shared__ uint32_t s_count[kSortWarps][kMaxBins];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
  for (int b = lane; b < bins; b += 32) s_count[warp][b] = 0;
  pdl_wait();
  __syncwarp();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kSortChunk + warp * (32 * kSortRounds) + lane;
  uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) key[r] = base + 32 * r < n ? source_key(src, base + 32 * r, nullptr) : 0u;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const bool ok = base + 32 * r < n;
    const uint32_t digit = (key[r] >> shift) & (bins - 1);
    const unsigned live = __ballot_sync(0xffffffffu, ok);
    const unsigned same = lanes_with(digit, bits, live);
    rank[r] = s_count[warp][digit] + __popc(same & ((1u << lane) - 1));
    __syncwarp();
    if (ok && (same >> lane) == 1u) s_count[warp][digit] += __popc(same);  // the last lane with it
    __syncwarp();
  }
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += kSortThreads) {
    uint32_t run = starts[static_cast<int64_t>(b) * chunks + blockIdx.x];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      const uint32_t q = s_count[w][b];
      s_count[w][b] = run;
      run += q;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = base + 32 * r;
    if (i >= n) continue;
    const uint32_t at = s_count[warp][(key[r] >> shift) & (bins - 1)] + rank[r];
    keys[at] = key[r];
    tokens[at] = src.ids != nullptr ? static_cast<uint32_t>(i) : src.tokens[i];
  }
}

// The whole sort by one cluster of up to 8 blocks, each with 1024 R tokens.  A pass ranks
// the tokens as above, adds up the blocks' counts out of their shared memory, and puts
// its tokens in order in shared memory first, so that neighbours then travel together to
// their places in the blocks' shared memory, in the last pass to global memory.
constexpr int kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32, kMaxCluster = 8, kMaxRounds = 8;
constexpr int64_t kClusterMost = int64_t(kMaxCluster) * kClusterThreads * kMaxRounds;

__device__ __forceinline__ uint32_t cluster_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_store(uint32_t a, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}
constexpr size_t cluster_sort_smem(int R) {
  return static_cast<size_t>(2 * R * kClusterThreads) * 8 + 2 * kMaxBins * 4 + kClusterWarps * kMaxBins * 2;
}

template <int R>
__global__ void __launch_bounds__(kClusterThreads) sort_cluster_kernel(const Source src, int n, int passes, int bits,
                                                                      uint32_t* __restrict__ keys,
                                                                      uint32_t* __restrict__ tokens, int* status) {
  constexpr int kLen = R * kClusterThreads;
  extern __shared__ uint64_t s_sort[];
  uint64_t* s_place = s_sort;          // [kLen] this block's places: key and token
  uint64_t* s_local = s_place + kLen;  // [kLen] this block's tokens in the pass's order
  uint32_t* s_total = reinterpret_cast<uint32_t*>(s_local + kLen);  // [bins] tokens of a bin in this block
  uint32_t* s_delta = s_total + kMaxBins;  // [bins] from a token's place in s_local to its place in all
  uint16_t* s_count = reinterpret_cast<uint16_t*>(s_delta + kMaxBins);  // [warps][bins]
  __shared__ uint32_t s_all[kMaxBins / 32], s_own[kMaxBins / 32], s_first[kMaxBins];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << bits;
  const int me = static_cast<int>(cluster_ctarank()), blocks = static_cast<int>(gridDim.x);
  const int have = min(kLen, max(0, n - me * kLen));
  const int first = warp * 32 * R + lane;  // of this thread's places in the block, 32 apart
  uint16_t* mine = s_count + warp * bins;
  pdl_wait();
  pdl_launch();
  uint32_t key[R], token[R], rank[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    token[r] = me * kLen + first + 32 * r;
    key[r] = first + 32 * r < have ? key_of(src.ids, src.id64, token[r], src.V, src.pad, status) : 0u;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * bits;
    if (p > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint64_t q = s_place[first + 32 * r];
        key[r] = static_cast<uint32_t>(q >> 32);
        token[r] = static_cast<uint32_t>(q);
      }
    }
    for (int b = lane; b < bins; b += 32) mine[b] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool ok = first + 32 * r < have;
      const uint32_t digit = (key[r] >> shift) & (bins - 1);
      const unsigned live = __ballot_sync(0xffffffffu, ok);
      const unsigned same = lanes_with(digit, bits, live);
      rank[r] = mine[digit] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (ok && (same >> lane) == 1u) mine[digit] = static_cast<uint16_t>(mine[digit] + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    uint32_t own = 0;  // tokens of bin threadIdx.x in this block
    if (static_cast<int>(threadIdx.x) < bins) {
#pragma unroll 16
      for (int w = 0; w < kClusterWarps; ++w) {
        const uint32_t q = s_count[w * bins + threadIdx.x];
        s_count[w * bins + threadIdx.x] = static_cast<uint16_t>(own);
        own += q;
      }
      s_total[threadIdx.x] = own;
    }
    if (blocks > 1) cluster_sync();
    uint32_t before = 0, all = own, all_incl = 0, own_incl = 0;
    if (static_cast<int>(threadIdx.x) < kMaxBins) {  // whole warps
      if (blocks > 1 && static_cast<int>(threadIdx.x) < bins) {
        all = 0;
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
          const uint32_t v = q < blocks ? cluster_load(mapa_shared(smem_u32(s_total + threadIdx.x), q)) : 0u;
          before += q < me ? v : 0u;
          all += v;
        }
      }
      all_incl = all;
      own_incl = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, all_incl, o), v = __shfl_up_sync(0xffffffffu, own_incl, o);
        if (lane >= o) all_incl += u, own_incl += v;
      }
      if (lane == 31) s_all[warp] = all_incl, s_own[warp] = own_incl;
    }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < bins) {
      for (int w = 0; w < warp; ++w) all_incl += s_all[w], own_incl += s_own[w];
      const uint32_t local = own_incl - own;  // first place of the bin in s_local
      s_delta[threadIdx.x] = all_incl - all + before - local;
      s_first[threadIdx.x] = local;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (first + 32 * r >= have) continue;
      const uint32_t digit = (key[r] >> shift) & (bins - 1);
      s_local[s_first[digit] + mine[digit] + rank[r]] = (static_cast<uint64_t>(key[r]) << 32) | token[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = threadIdx.x + r * kClusterThreads;
      if (i >= have) continue;
      const uint64_t q = s_local[i];
      const uint32_t at = i + s_delta[(static_cast<uint32_t>(q >> 32) >> shift) & (bins - 1)];
      if (p == passes - 1) {
        keys[at] = static_cast<uint32_t>(q >> 32);
        tokens[at] = static_cast<uint32_t>(q);
      } else if (blocks > 1) {
        cluster_store(mapa_shared(smem_u32(s_place + at % kLen), at / kLen), q);
      } else {
        s_place[at] = q;
      }
    }
    // every place is filled, and every block has read the counts
    if (blocks > 1) cluster_sync();
    else __syncthreads();
  }
}

// ---- sums --------------------------------------------------------------------
// Blocks of 16 KB in the order of their addresses: 1.24 GB in 162 us (7.7 TB/s), where
// blocks that walk the whole range in turn take 175 to 195.
constexpr int kZeroThreads = 256, kZeroWords = 4, kZeroBlock = kZeroThreads * kZeroWords;  // 16-byte words
// `beside`: launched while the sort runs, whose results it does not touch; one block waits
// for the sort at its end, so that what waits for this kernel has waited for both (all
// blocks would hold their places on the SMs until then).
__global__ void __launch_bounds__(kZeroThreads) embed_zero_kernel(uint8_t* __restrict__ p, int64_t bytes, int head,
                                                                 bool beside) {
  if (!beside) pdl_wait();
  // p + head is 16-byte aligned; bytes counts from p
  const int64_t words = (bytes - head) / 16;
  uint4* w = reinterpret_cast<uint4*>(p + head);
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kZeroBlock + threadIdx.x;
#pragma unroll
  for (int u = 0; u < kZeroWords; ++u)
    if (i0 + u * kZeroThreads < words) w[i0 + u * kZeroThreads] = make_uint4(0u, 0u, 0u, 0u);
  if (blockIdx.x == 0) {
    if (static_cast<int>(threadIdx.x) < head) p[threadIdx.x] = 0;
    const int64_t rest = head + words * 16 + threadIdx.x;
    if (threadIdx.x < 16 && rest < bytes) p[rest] = 0;
  }
  if (beside && blockIdx.x == 0) pdl_wait();
}

// One bit for each row of the table that a token names; a block has kMarkRows rows.
constexpr int kMarkRows = 1 << 18;
__global__ void __launch_bounds__(1024) embed_mark_kernel(const Source src, int n, uint32_t* __restrict__ named) {
  __shared__ uint32_t s_named[kMarkRows / 32];
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * kMarkRows;
  const int rows = static_cast<int>(min(static_cast<int64_t>(kMarkRows), src.V - v0)), words = (rows + 31) / 32;
  for (int i = threadIdx.x; i < words; i += 1024) s_named[i] = 0;
  pdl_wait();
  __syncthreads();
  for (int t = threadIdx.x; t < n; t += 1024) {
    const int64_t r = static_cast<int64_t>(key_of(src.ids, src.id64, t, src.V, src.pad, nullptr)) - v0;
    if (r >= 0 && r < rows) atomicOr(&s_named[r >> 5], 1u << (r & 31));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < words; i += 1024) named[v0 / 32 + i] = s_named[i];
}

// Zeros for the rows without a token (`named`, complete before the sort began), beside
// the sort, the sums and the joins of a small batch, which write the others.  It is
// launched last, while those wait for one another, and a block waits for them at its end.
// As it has not waited for the marks' launch itself, it reads them from the L2.
// Rows of whole words on 16-byte boundaries: a block takes `each` rows, about 16 KB, and
// mostly finds none of them named.
__global__ void __launch_bounds__(kZeroThreads) embed_zero_whole_rows_kernel(const uint32_t* __restrict__ named,
                                                                            uint4* __restrict__ p, int64_t V,
                                                                            int each, int row_words) {
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * each;
  const int rows = static_cast<int>(min(static_cast<int64_t>(each), V - row0));
  auto is_named = [&](int64_t r) { return __ldcg(named + (r >> 5)) >> (r & 31) & 1u; };
  bool any = false;
  for (int r = threadIdx.x; r < rows; r += kZeroThreads) any |= is_named(row0 + r) != 0;
  uint4* w = p + row0 * row_words;
  const int words = rows * row_words;
  if (!__syncthreads_or(any)) {
#pragma unroll 4
    for (int i = threadIdx.x; i < words; i += kZeroThreads) w[i] = make_uint4(0u, 0u, 0u, 0u);
  } else {
    for (int i = threadIdx.x; i < words; i += kZeroThreads)
      if (!is_named(row0 + i / row_words)) w[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  if (blockIdx.x == 0) pdl_wait();
}

// The same for rows that begin anywhere, by the words of the whole table.  A word holds
// values of two rows at most where a row has its 16 bytes; narrower rows are looked up
// value by value.
__global__ void __launch_bounds__(kZeroThreads) embed_zero_rows_kernel(const uint32_t* __restrict__ named,
                                                                      uint8_t* __restrict__ p, int64_t bytes,
                                                                      int head, unsigned row_bytes, int size) {
  // the words of the block, from the 16-byte aligned p + head on, and the row it begins in
  const int64_t from = static_cast<int64_t>(blockIdx.x) * kZeroBlock * 16 + head;
  const int64_t row0 = from / row_bytes;
  const unsigned off0 = static_cast<unsigned>(from - row0 * row_bytes);
  const bool wide = row_bytes >= 16;
  auto is_named = [&](int64_t r) { return __ldcg(named + (r >> 5)) >> (r & 31) & 1u; };
#pragma unroll
  for (int u = 0; u < kZeroWords; ++u) {
    const unsigned at = 16u * (threadIdx.x + u * kZeroThreads);
    if (from + at + 16 > bytes) continue;
    const int64_t r = row0 + (off0 + at) / row_bytes, q = row0 + (off0 + at + 15) / row_bytes;
    const bool a = is_named(r), b = q != r && is_named(q);
    if (wide && !a && !b) {
      *reinterpret_cast<uint4*>(p + from + at) = make_uint4(0u, 0u, 0u, 0u);
    } else if (!wide || (q != r && !(a && b))) {
      for (unsigned e = 0; e < 16; e += size)
        if (!is_named(row0 + (off0 + at + e) / row_bytes)) {
          if (size == 2) *reinterpret_cast<uint16_t*>(p + from + at + e) = 0;
          else *reinterpret_cast<uint32_t*>(p + from + at + e) = 0u;
        }
    }
  }
  if (blockIdx.x == 0) {  // the bytes before the first word and after the last
    const int64_t rest = head + (bytes - head) / 16 * 16 + threadIdx.x;
    if (static_cast<int>(threadIdx.x) < head && !is_named(threadIdx.x / row_bytes)) p[threadIdx.x] = 0;
    if (threadIdx.x < 16 && rest < bytes && !is_named(rest / row_bytes)) p[rest] = 0;
    pdl_wait();
  }
}

struct SumArgs {
  const void* dout;
  void* dtable;
  const uint32_t *keys, *tokens;
  float* part;          // [chunks][2][ld]
  int64_t T, chunks;
  int V, d, ld, len;    // len: tokens of a chunk
  int width, tiles;     // shares of a tile of columns (threads of a group), tiles of a row
  int groups;           // chunks of a block
  float scale;
  int add;
  int early;            // lets the next kernel start at once: a small batch's launches wait side by side
};

// Columns 8 v .. 8 v + 7 of a row that begins anywhere: the two or three aligned words
// that hold them, shifted into place.  Words that reach past the whole tensor
// [begin, end) are read value by value; columns past d are 0.
__device__ __forceinline__ uint4 word_within(uintptr_t w, uintptr_t begin, uintptr_t end, bf16_t) {
  if (w >= begin && w + 16 <= end) return *reinterpret_cast<const uint4*>(w);
  uint32_t q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uintptr_t p = w + 2 * e;
    q[e] = p >= begin && p < end ? *reinterpret_cast<const uint16_t*>(p) : 0u;
  }
  return make_uint4(q[0] | q[1] << 16, q[2] | q[3] << 16, q[4] | q[5] << 16, q[6] | q[7] << 16);
}
__device__ __forceinline__ float4 word_within(uintptr_t w, uintptr_t begin, uintptr_t end, float) {
  if (w >= begin && w + 16 <= end) return *reinterpret_cast<const float4*>(w);
  float q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uintptr_t p = w + 4 * e;
    q[e] = p >= begin && p < end ? *reinterpret_cast<const float*>(p) : 0.f;
  }
  return make_float4(q[0], q[1], q[2], q[3]);
}
__device__ __forceinline__ void load8_any(const bf16_t* row, int v, int d, uintptr_t begin, uintptr_t end,
                                          Raw8<bf16_t>& r) {
  r.v = make_uint4(0u, 0u, 0u, 0u);
  if (8 * v >= d) return;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + 8 * v), word = at & ~uintptr_t(15);
  const unsigned shift = static_cast<unsigned>(at - word) / 2;  // values
  const uint4 a = word_within(word, begin, end, bf16_t{});
  uint4 b = make_uint4(0u, 0u, 0u, 0u);
  if (shift != 0 && word + 16 < end) b = word_within(word + 16, begin, end, bf16_t{});
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (shift & 4)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (shift & 2)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  if (shift & 1)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  const int left = d - 8 * v;  // columns that are the row's
  if (left < 8)
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= left >= 2 * i + 2 ? 0xFFFFFFFFu : left == 2 * i + 1 ? 0xFFFFu : 0u;
  r.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load8_any(const float* row, int v, int d, uintptr_t begin, uintptr_t end,
                                          Raw8<float>& r) {
  r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (8 * v >= d) return;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row + 8 * v), word = at & ~uintptr_t(15);
  const unsigned shift = static_cast<unsigned>(at - word) / 4;
  const float4 a = word_within(word, begin, end, 0.f);
  float4 b = make_float4(0.f, 0.f, 0.f, 0.f), c = b;
  if (word + 16 < end) b = word_within(word + 16, begin, end, 0.f);
  if (shift != 0 && word + 32 < end) c = word_within(word + 32, begin, end, 0.f);
  float w[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
  if (shift & 2)
#pragma unroll
    for (int i = 0; i < 10; ++i) w[i] = w[i + 2];
  if (shift & 1)
#pragma unroll
    for (int i = 0; i < 9; ++i) w[i] = w[i + 1];
  const int left = d - 8 * v;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = i < left ? w[i] : 0.f;
  r.a = make_float4(w[0], w[1], w[2], w[3]);
  r.b = make_float4(w[4], w[5], w[6], w[7]);
}

// Adds scale * f (or writes it) to columns 8 v .. 8 v + 7 of row `key`.  Not VEC: whole
// warps call this, 32 shares in a row each, and pass the 256 columns through shared
// memory (turn: 256 floats of the warp), so that neighbouring lanes write neighbouring
// values.
template <typename G, bool VEC>
__device__ __forceinline__ void put_row(const SumArgs& a, uint32_t key, int v, const f2 (&f)[4], float* turn) {
  G* row = static_cast<G*>(a.dtable) + static_cast<int64_t>(key) * a.d;
  const f2 s = pk(a.scale);
  f2 r[4], g[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) g[e] = f[e];
  if (!VEC) {
    const int lane = threadIdx.x & 31;
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(turn + 8 * lane + 2 * e) = unpk(f[e]);
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = pk(turn[lane + 64 * e], turn[lane + 64 * e + 32]);
  }
  if (a.add) {
    get8<G, VEC>(row, v, a.d, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = fma2(g[e], s, r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = mul2(g[e], s);
  }
  put8<G, VEC>(row, v, a.d, r);
}
__device__ __forceinline__ float* part_row(const SumArgs& a, int64_t chunk, int last) {
  return a.part + (2 * chunk + last) * a.ld;
}

// Rows whose loads are in flight: 128 bytes a thread, four rows where each takes two or
// three aligned words (30011 x 1001 added: 72 us, with eight rows 87).
template <typename T>
constexpr int kAhead = 16 / sizeof(T);
constexpr int kMaxLen = 64, kMaxGroups = 32;
template <typename T, typename G, bool VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs a) {
  __shared__ uint32_t s_key[kMaxGroups * kMaxLen], s_token[kMaxGroups * kMaxLen];
  __shared__ float s_turn[VEC ? 1 : 8 * 256];
  const int group = threadIdx.x / a.width;
  const uint32_t none = static_cast<uint32_t>(a.V);
  float* turn = s_turn + (VEC ? 0 : (threadIdx.x >> 5) * 256);
  if (a.early) pdl_launch();
  pdl_wait();
  // the chunks' ids and tokens, all at once
  for (int i = threadIdx.x; i < a.groups * a.len; i += blockDim.x) {
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * a.groups + i / a.len) / a.tiles * a.len + i % a.len;
    s_key[i] = at < a.T ? a.keys[at] : none;
    s_token[i] = at < a.T ? a.tokens[at] : 0u;
  }
  const int64_t item = static_cast<int64_t>(blockIdx.x) * a.groups + group, chunk = item / a.tiles;
  const int v = static_cast<int>(item - chunk * a.tiles) * a.width + threadIdx.x - group * a.width;
  const int64_t i0 = chunk * a.len;
  const bool live = i0 < a.T && (!VEC || 8 * v < a.d);
  const uint32_t prev = live && i0 > 0 ? a.keys[i0 - 1] : none, next = live && i0 + a.len < a.T ? a.keys[i0 + a.len] : none;
  __syncthreads();
  if (!live) return;
  const uint32_t *keys = s_key + group * a.len, *tokens = s_token + group * a.len;
  uint32_t key = keys[0];
  if (key == none) return;
  bool open = prev == key;  // the run that this chunk begins with began before it
  f2 sum[4] = {pk(0.f), pk(0.f), pk(0.f), pk(0.f)};
  const T* dout = static_cast<const T*>(a.dout);
  const uintptr_t begin = reinterpret_cast<uintptr_t>(dout), end = reinterpret_cast<uintptr_t>(dout + a.T * a.d);
  constexpr int A = VEC ? kAhead<T> : 4;
  for (int i = 0; i < a.len; i += A) {
    Raw8<T> raw[A];
#pragma unroll
    for (int u = 0; u < A; ++u)
      if (keys[i + u] != none) {
        const T* row = dout + static_cast<int64_t>(tokens[i + u]) * a.d;
        if (VEC) load8<true>(row, v, a.d, raw[u]);
        else load8_any(row, v, a.d, begin, end, raw[u]);
      }
#pragma unroll
    for (int u = 0; u < A; ++u) {
      const uint32_t k = keys[i + u];
      if (k != key) {
        if (open) put8<float, true>(part_row(a, chunk, 0), v, a.ld, sum);
        else put_row<G, VEC>(a, key, v, sum, turn);
        open = false;
        key = k;
        if (key == none) return;
        sum[0] = sum[1] = sum[2] = sum[3] = pk(0.f);
      }
      f2 f[4];
      widen(raw[u], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], f[e]);
    }
  }
  if (open) put8<float, true>(part_row(a, chunk, 0), v, a.ld, sum);
  else if (next == key) put8<float, true>(part_row(a, chunk, 1), v, a.ld, sum);
  else put_row<G, VEC>(a, key, v, sum, turn);
}

// Runs that reach over chunk borders.  The chunk that a run begins in adds its own part
// and the first parts of the chunks that follow, up to the one the run ends in.  A block
// looks at 16 chunks, a lane each (4096 x 2048 added: 34 us, with 32 chunks 36); a warp
// takes 256 columns of a short run by itself, the eight warps every eighth part of a long
// one, whose sums warp 0 then adds.
constexpr int kJoinChunks = 16, kLongRun = 32;
template <typename G, bool VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumArgs a) {
  __shared__ float s_sum[8][256];
  __shared__ uint32_t s_key[kJoinChunks], s_first[256];
  __shared__ int64_t s_parts[kJoinChunks];  // parts of the run that begins in a chunk, 0: none to add
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (a.early) pdl_launch();
  pdl_wait();
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kJoinChunks;
  const uint32_t none = static_cast<uint32_t>(a.V);
  // the first ids of this block's chunks and of those that follow, all at once
  s_first[threadIdx.x] = c0 + threadIdx.x < a.chunks ? a.keys[(c0 + threadIdx.x) * a.len] : none;
  uint32_t key = none, prev = none;
  const int64_t chunk = c0 + lane, i0 = chunk * a.len;
  if (warp == 0 && lane < kJoinChunks && chunk < a.chunks - 1) {
    key = a.keys[i0 + a.len - 1];
    if (i0 > 0) prev = a.keys[i0 - 1];
  }
  __syncthreads();
  if (warp == 0 && lane < kJoinChunks) {
    int64_t parts = 0;
    if (key != none && s_first[lane + 1] == key && !(s_first[lane] == key && prev == key)) {
      // the last chunk with a part of the run: within reach, or by bisection over first ids
      int near = lane + 1;
#pragma unroll
      for (int step = 128; step > 0; step >>= 1)
        if (near + step < 256 && s_first[near + step] == key) near += step;
      int64_t lo = c0 + near, hi = near < 255 ? lo : a.chunks - 1;
      while (lo < hi) {
        const int64_t mid = (lo + hi + 1) / 2;
        if (a.keys[mid * a.len] == key) lo = mid;
        else hi = mid - 1;
      }
      parts = lo - chunk + 1;
    }
    s_key[lane] = key;
    s_parts[lane] = parts;
  }
  __syncthreads();
  const int v = blockIdx.y * 32 + lane;
  auto add_parts = [&](int64_t chunk, int64_t parts, int64_t from, int64_t step, f2 (&sum)[4]) {
    sum[0] = sum[1] = sum[2] = sum[3] = pk(0.f);
    for (int64_t q = from; q < parts; q += 4 * step) {
      Raw8<float> raw[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t p = q + u * step;
        if (p < parts) load8<true>(part_row(a, chunk + p, p == 0 ? 1 : 0), v, a.ld, raw[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (q + u * step >= parts) break;
        f2 f[4];
        widen(raw[u], f);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], f[e]);
      }
    }
  };
  f2 sum[4];
  for (int i = warp; i < kJoinChunks; i += 8) {
    const int64_t parts = s_parts[i];
    if (parts == 0 || parts > kLongRun) continue;
    add_parts(c0 + i, parts, 0, 1, sum);
    put_row<G, VEC>(a, s_key[i], v, sum, s_sum[warp]);
  }
  for (int i = 0; i < kJoinChunks; ++i) {
    const int64_t parts = s_parts[i];
    if (parts <= kLongRun) continue;
    add_parts(c0 + i, parts, warp, 8, sum);
    __syncthreads();  // s_sum was read
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(&s_sum[warp][64 * e + 2 * lane]) = unpk(sum[e]);
    __syncthreads();
    if (warp != 0) continue;
    for (int w = 1; w < 8; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = *reinterpret_cast<const float2*>(&s_sum[w][64 * e + 2 * lane]);
        sum[e] = add2(sum[e], pk(x.x, x.y));
      }
    put_row<G, VEC>(a, s_key[i], v, sum, s_sum[0]);
  }
}

// ---- sizes -------------------------------------------------------------------
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tokens of a chunk, a multiple of 8: 8 or 16 where the chunks then run at once, three
// blocks of 256 threads with 8 columns each on an SM; 16 up to 32768 tokens of any width
// (30011 x 1001 added 70 us, with 24 or 32 80 to 83; x 2048 81, 78; 20000 x 1500 71, 80); else
// 32 or, past 131072 tokens, 64 (kMaxLen), for fewer parts.
int chunk_len(int64_t T, int64_t d) {
  const int64_t at_once = 3 * kSMs * 2048;
  return T * d <= 8 * at_once ? 8 : T * d <= 16 * at_once || T <= 32768 ? 16 : T <= 131072 ? 32 : 64;
}

// Whether a dense gradient's zeros are written beside everything else: for a batch whose
// sums fit the SMs at once with room left.  (Then all that stands before the zeros is a
// launch that marks the tokens' rows; else they are written beside the sort.)
constexpr int kBesideTokens = 8192;
bool zeros_beside(int64_t T, int64_t d) { return T <= kBesideTokens && T * d <= int64_t(16) * 2 * kSMs * 2048; }

struct Workspace {
  uint32_t *keys[2], *tokens[2], *counts, *named;
  float* part;
  size_t bytes;
};
Workspace workspace(void* ws, int64_t T, int V, int d) {
  Workspace q = {};
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = p + at;
    at += static_cast<size_t>(round_up(static_cast<int64_t>(bytes), 256));
    return r;
  };
  const int64_t sort_chunks = (T + kSortChunk - 1) / kSortChunk;
  for (int i = 0; i < 2; ++i) {
    q.keys[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(T) * 4));
    q.tokens[i] = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(T) * 4));
  }
  q.counts = reinterpret_cast<uint32_t*>(take((static_cast<size_t>(sort_chunks) << digits(V).bits) * 4));
  q.named = reinterpret_cast<uint32_t*>(take(zeros_beside(T, d) ? (static_cast<size_t>(V) + 31) / 32 * 4 : 0));
  const int64_t len = chunk_len(T, d), chunks = (T + len - 1) / len;
  q.part = reinterpret_cast<float*>(take(static_cast<size_t>(chunks) * 2 * static_cast<size_t>(round_up(d, 8)) * 4));
  q.bytes = at;
  return q;
}

// ---- launches ----------------------------------------------------------------
template <typename T, typename O, int SH>
cudaError_t forward(const moe_embed_desc* q, bool vec, const void* ids, const void* table, void* out, int* status,
                    cudaStream_t s) {
  const int64_t segs = (static_cast<int64_t>(q->d) + 256 * SH - 1) / (256 * SH);
  const int64_t blocks = (q->T * segs + kFwdWarps - 1) / kFwdWarps;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(vec ? embed_fwd_kernel<T, O, true, SH> : embed_fwd_kernel<T, O, false, SH>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kFwdThreads), 0, s, ids,
                    q->id_type == MOE_I64 ? 1 : 0, static_cast<const T*>(table), static_cast<int64_t>(q->T), q->V,
                    q->d, q->scale, static_cast<O*>(out), (reinterpret_cast<uintptr_t>(out) & 31u) == 0, status);
}
template <typename T, typename O>
cudaError_t forward(const moe_embed_desc* q, bool vec, const void* ids, const void* table, void* out, int* status,
                    cudaStream_t s) {
  return static_cast<int64_t>(q->T) * ((q->d + 1023) / 1024) >= 64 * kSMs
             ? forward<T, O, 4>(q, vec, ids, table, out, status, s)
             : forward<T, O, 2>(q, vec, ids, table, out, status, s);
}

int head_of(const void* p, int64_t bytes) {  // bytes before the first 16-byte boundary
  return static_cast<int>(std::min<int64_t>(static_cast<int64_t>(-reinterpret_cast<intptr_t>(p) & 15), bytes));
}
int64_t zero_blocks(int64_t bytes) { return bytes / (16 * kZeroBlock) + 1; }
cudaError_t zeros(void* p, int64_t bytes, bool beside, cudaStream_t s) {
  if (zero_blocks(bytes) > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(embed_zero_kernel, dim3(static_cast<unsigned>(zero_blocks(bytes))), dim3(kZeroThreads), 0, s,
                    static_cast<uint8_t*>(p), bytes, head_of(p, bytes), beside);
}
cudaError_t mark_rows(const Source& src, int n, uint32_t* named, cudaStream_t s) {
  return launch_pdl(embed_mark_kernel, dim3(static_cast<unsigned>((static_cast<int64_t>(src.V) + kMarkRows - 1) / kMarkRows)),
                    dim3(1024), 0, s, src, n, named);
}
cudaError_t zero_rows(const uint32_t* named, void* p, int64_t V, int64_t d, unsigned size, cudaStream_t s) {
  const int64_t bytes = V * d * size, row_bytes = d * size;
  if (row_bytes % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
    const int64_t each = std::max<int64_t>(1, 16 * kZeroBlock / row_bytes), blocks = (V + each - 1) / each;
    return launch_pdl(embed_zero_whole_rows_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kZeroThreads), 0, s,
                      named, static_cast<uint4*>(p), V, static_cast<int>(each), static_cast<int>(row_bytes / 16));
  }
  if (zero_blocks(bytes) > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(embed_zero_rows_kernel, dim3(static_cast<unsigned>(zero_blocks(bytes))), dim3(kZeroThreads), 0, s,
                    named, static_cast<uint8_t*>(p), bytes, head_of(p, bytes), static_cast<unsigned>(d * size),
                    static_cast<int>(size));
}

template <int R>
cudaError_t sort_cluster(const Source& src, const moe_embed_desc* q, const Workspace& w, unsigned blocks, int* status,
                         cudaStream_t s) {
  const Digits g = digits(q->V);
  const cudaError_t e = cudaFuncSetAttribute(sort_cluster_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(cluster_sort_smem(R)));
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(sort_cluster_kernel<R>, dim3(blocks), dim3(kClusterThreads), cluster_sort_smem(R), s, blocks,
                            src, q->T, g.passes, g.bits, w.keys[0], w.tokens[0], status);
}

// Sorts the tokens by id; the result is in keys[*out], tokens[*out].
cudaError_t sort_tokens(const moe_embed_desc* q, const void* ids, int64_t pad, const Workspace& w, int* status,
                        int* out, cudaStream_t s) {
  const Digits g = digits(q->V);
  const int bins = 1 << g.bits;
  const int64_t n = q->T, chunks = (n + kSortChunk - 1) / kSortChunk;
  Source src = {ids, nullptr, nullptr, q->id_type == MOE_I64 ? 1 : 0, q->V, pad};
  if (n <= kClusterMost) {
    // as many blocks as have 1024 tokens each, then more tokens to a block
    unsigned blocks = 1;
    while (blocks < kMaxCluster && static_cast<int64_t>(blocks) * kClusterThreads < n) blocks *= 2;
    const int64_t rounds = (n + static_cast<int64_t>(blocks) * kClusterThreads - 1) / (static_cast<int64_t>(blocks) * kClusterThreads);
    *out = 0;
    return rounds <= 1   ? sort_cluster<1>(src, q, w, blocks, status, s)
           : rounds <= 2 ? sort_cluster<2>(src, q, w, blocks, status, s)
           : rounds <= 4 ? sort_cluster<4>(src, q, w, blocks, status, s)
                         : sort_cluster<8>(src, q, w, blocks, status, s);
  }
  cudaError_t e = cudaSuccess;
  for (int p = 0; p < g.passes && e == cudaSuccess; ++p) {
    const int shift = p * g.bits, to = p & 1;
    e = launch_pdl(sort_count_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kSortThreads), 0, s, src, n, shift,
                   bins, static_cast<int>(chunks), w.counts, p == 0 ? status : nullptr);
    if (e != cudaSuccess) break;
    e = launch_pdl(sort_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, w.counts, chunks * bins);
    if (e != cudaSuccess) break;
    e = launch_pdl(sort_place_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kSortThreads), 0, s, src, n, shift,
                   g.bits, static_cast<int>(chunks), static_cast<const uint32_t*>(w.counts), w.keys[to], w.tokens[to]);
    src.ids = nullptr;
    src.keys = w.keys[to];
    src.tokens = w.tokens[to];
    *out = to;
  }
  return e;
}

template <typename T, typename G, bool VEC>
cudaError_t sums(SumArgs a, cudaStream_t s) {
  // shares of a row: whole vectors, or warps of 256 columns
  const int shares = VEC ? (a.d + 7) / 8 : static_cast<int>((static_cast<int64_t>(a.d) + 255) / 256 * 32);
  a.tiles = (shares + 255) / 256;
  a.width = (shares + a.tiles - 1) / a.tiles;
  if (!VEC) a.width = (a.width + 31) / 32 * 32;
  a.groups = std::min(kMaxGroups, 256 / a.width);
  const int64_t items = a.chunks * a.tiles, blocks = (items + a.groups - 1) / a.groups;
  cudaError_t e = launch_pdl(embed_sum_kernel<T, G, VEC>, dim3(static_cast<unsigned>(blocks)),
                             dim3(static_cast<unsigned>(a.width * a.groups)), 0, s, a);
  if (e != cudaSuccess || a.chunks < 2) return e;
  return launch_pdl(embed_join_kernel<G, VEC>,
                    dim3(static_cast<unsigned>((a.chunks - 1 + kJoinChunks - 1) / kJoinChunks),
                         static_cast<unsigned>((static_cast<int64_t>(a.d) + 255) / 256)),
                    dim3(256), 0, s, a);
}
template <typename T, typename G>
cudaError_t sums(const SumArgs& a, bool vec, cudaStream_t s) {
  return vec ? sums<T, G, true>(a, s) : sums<T, G, false>(a, s);
}

int bad(const char* msg) { return record_error(MOE_ERR_INVALID_ARG, msg); }
bool misaligned(const void* p, unsigned size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; }
bool is_type(int t) { return t == MOE_F32 || t == MOE_BF16; }
unsigned size_of(int t) { return t == MOE_BF16 ? 2u : 4u; }

constexpr int kMaxD = 1 << 20;  // the join's grid; more columns than any table has

int check_desc(const moe_embed_desc* q) {
  if (q == nullptr) return bad("desc is NULL");
  if (q->T < 0 || q->V <= 0 || q->d <= 0) return bad("T must not be negative, V and d must be positive");
  if (q->d > kMaxD) return record_error(MOE_ERR_UNSUPPORTED, "d > 2^20");
  if (q->id_type != MOE_I32 && q->id_type != MOE_I64) return bad("id_type must be MOE_I32 or MOE_I64");
  if (!is_type(q->table_type) || !is_type(q->row_type)) return bad("table_type and row_type must be MOE_F32 or MOE_BF16");
  if (!std::isfinite(q->scale)) return bad("scale must be finite");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_embed_fwd(const moe_embed_desc* desc, const void* ids, const void* table, void* out, moe_stream_t stream) {
  NvtxScope nvtx("moe_embed_fwd");
  int rc = check_desc(desc);
  if (rc) return rc;
  if (desc->T == 0) return record_error(MOE_OK, "");
  if (!ids || !table || !out) return bad("NULL pointer");
  if (misaligned(ids, desc->id_type == MOE_I64 ? 8 : 4) || misaligned(table, size_of(desc->table_type)) ||
      misaligned(out, size_of(desc->row_type)))
    return bad("misaligned pointer");
  int* status = nullptr;
  rc = device_status_word(&status);
  if (rc != MOE_OK) return rc;
  const bool vec = desc->d % 8 == 0 && !misaligned(table, 16) && !misaligned(out, 16);
  ProbeScope probe("embed_fwd", stream);
  cudaError_t e;
  if (desc->table_type == MOE_BF16)
    e = desc->row_type == MOE_BF16 ? forward<bf16_t, bf16_t>(desc, vec, ids, table, out, status, stream)
                                   : forward<bf16_t, float>(desc, vec, ids, table, out, status, stream);
  else
    e = desc->row_type == MOE_BF16 ? forward<float, bf16_t>(desc, vec, ids, table, out, status, stream)
                                   : forward<float, float>(desc, vec, ids, table, out, status, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

size_t moe_embed_workspace_size(int32_t T, int32_t V, int32_t d) {
  if (T <= 0 || V <= 0 || d <= 0 || d > kMaxD) return 0;
  return workspace(nullptr, T, V, d).bytes;
}

int moe_embed_bwd(const moe_embed_desc* desc, const void* ids, const void* dout, void* dtable, int64_t pad_id,
                  int32_t accumulate, void* ws, size_t ws_bytes, moe_stream_t stream) {
  NvtxScope nvtx("moe_embed_bwd");
  int rc = check_desc(desc);
  if (rc) return rc;
  if (accumulate != 0 && accumulate != 1) return bad("accumulate must be 0 or 1");
  const bool any = desc->T > 0;
  if (!dtable || misaligned(dtable, size_of(desc->table_type))) return bad("dtable NULL or misaligned");
  if (any) {
    if (!ids || !dout || !ws) return bad("NULL pointer");
    if (misaligned(ids, desc->id_type == MOE_I64 ? 8 : 4) || misaligned(dout, size_of(desc->row_type)) ||
        misaligned(ws, 16))
      return bad("misaligned pointer");
    if (ws_bytes < moe_embed_workspace_size(desc->T, desc->V, desc->d))
      return record_error(MOE_ERR_WORKSPACE, "embedding workspace too small");
  }
  int* status = nullptr;
  rc = device_status_word(&status);
  if (rc != MOE_OK) return rc;
  ProbeScope probe("embed_bwd", stream);
  cudaError_t e = cudaSuccess;
  Workspace w = {};
  int at = 0;
  const bool beside = any && !accumulate && zeros_beside(desc->T, desc->d);
  const Source src = {ids, nullptr, nullptr, desc->id_type == MOE_I64 ? 1 : 0, desc->V, pad_id};
  if (any) {
    w = workspace(ws, desc->T, desc->V, desc->d);
    if (beside) e = mark_rows(src, desc->T, w.named, stream);
  }
  if (any && e == cudaSuccess) {
    e = sort_tokens(desc, ids, pad_id, w, status, &at, stream);
  }
  if (!accumulate && !beside && e == cudaSuccess)
    e = zeros(dtable, static_cast<int64_t>(desc->V) * desc->d * size_of(desc->table_type),
              any && desc->T <= kClusterMost, stream);
  if (any && e == cudaSuccess) {
    SumArgs a = {};
    a.dout = dout; a.dtable = dtable; a.keys = w.keys[at]; a.tokens = w.tokens[at]; a.part = w.part;
    a.T = desc->T; a.len = chunk_len(desc->T, desc->d); a.chunks = (a.T + a.len - 1) / a.len;
    a.V = desc->V; a.d = desc->d; a.ld = static_cast<int>(round_up(desc->d, 8));
    a.scale = desc->scale; a.add = accumulate; a.early = beside;
    const bool vec = desc->d % 8 == 0 && !misaligned(dout, 16) && !misaligned(dtable, 16);
    if (desc->row_type == MOE_BF16)
      e = desc->table_type == MOE_BF16 ? sums<bf16_t, bf16_t>(a, vec, stream) : sums<bf16_t, float>(a, vec, stream);
    else
      e = desc->table_type == MOE_BF16 ? sums<float, bf16_t>(a, vec, stream) : sums<float, float>(a, vec, stream);
    if (beside && e == cudaSuccess) e = zero_rows(w.named, dtable, desc->V, desc->d, size_of(desc->table_type), stream);
  }
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
