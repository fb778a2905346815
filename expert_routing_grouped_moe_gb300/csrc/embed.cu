// Rows of a table for token ids, and the table's gradient.
//   out[t] = scale table[ids[t]]
//   dtable[v] = scale sum_{t: ids[t] = v} dout[t]     (dense, or added)
// Forward: a copy of rows, bound by memory.
//
// Gradient.  The tokens are sorted by id: a stable radix sort, least digit first,
// of up to 9 bits a pass, so two passes for a table of up to 2^18 rows.  Sorted
// tokens are cut into chunks of equal length, and a group of threads walks one
// chunk with 8 columns a thread: it adds up rows while the id stays the same and
// writes a run that lies in its chunk straight to the table.  A run that reaches
// over chunk borders leaves its parts in the workspace, [chunk][first, last], and
// a second kernel adds them in order.  So the work is even whatever the ids'
// frequencies, nothing is atomic, and the order of every sum depends on the ids
// alone.  What bounds it: T d reads of gradient rows and, dense, V d writes of
// which most are zeros.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

// ---- forward -----------------------------------------------------------------
// A warp moves up to 512 columns of a row, two shares of 8 a lane.
constexpr int kFwdThreads = 256, kFwdShares = 64;

template <typename T, typename O, bool VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const void* __restrict__ ids, int id64,
                                                               const T* __restrict__ table, int64_t T_, int V,
                                                               int d, float scale, O* __restrict__ out,
                                                               int* status) {
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int segs = (d + 8 * kFwdShares - 1) / (8 * kFwdShares);
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kFwdThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / segs;
  if (t >= T_) return;
  const int v0 = static_cast<int>(unit - t * segs) * kFwdShares + lane;
  const int64_t id = id64 ? static_cast<const int64_t*>(ids)[t] : static_cast<const int32_t*>(ids)[t];
  const bool ok = id >= 0 && id < V;
  if (!ok && lane == 0) atomicCAS(status, 0, kErrBadIds);
  const T* from = table + (ok ? id : 0) * static_cast<int64_t>(d);
  O* to = out + t * d;
  f2 f[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i) get8<T, VEC>(from, v0 + 32 * i, d, f[i]);
  const f2 s = pk(scale);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[i][e] = ok ? mul2(f[i][e], s) : pk(0.f);
    put8<O, VEC>(to, v0 + 32 * i, d, f[i]);
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
__global__ void __launch_bounds__(kSortThreads) sort_place_kernel(const Source src, int64_t n, int shift, int bins,
                                                                 int chunks, const uint32_t* __restrict__ starts,
                                                                 uint32_t* __restrict__ keys,
                                                                 uint32_t* __restrict__ tokens) {
  __shared__ uint32_t s_count[kSortWarps][kMaxBins];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
    const unsigned same = __match_any_sync(0xffffffffu, digit) & live;
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

// ---- sums --------------------------------------------------------------------
__global__ void __launch_bounds__(256) embed_zero_kernel(uint8_t* __restrict__ p, int64_t bytes, int head) {
  pdl_wait();
  // p + head is 16-byte aligned; bytes counts from p
  const int64_t words = (bytes - head) / 16;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  uint4* w = reinterpret_cast<uint4*>(p + head);
  for (int64_t i = i0; i < words; i += step) __stcs(w + i, make_uint4(0u, 0u, 0u, 0u));
  if (blockIdx.x == 0) {
    if (static_cast<int>(threadIdx.x) < head) p[threadIdx.x] = 0;
    const int64_t rest = head + words * 16 + threadIdx.x;
    if (threadIdx.x < 16 && rest < bytes) p[rest] = 0;
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
};

// Adds scale * f (or writes it) to row `key`, share v.
template <typename G, bool VEC>
__device__ __forceinline__ void put_row(const SumArgs& a, uint32_t key, int v, const f2 (&f)[4]) {
  G* row = static_cast<G*>(a.dtable) + static_cast<int64_t>(key) * a.d;
  const f2 s = pk(a.scale);
  f2 r[4];
  if (a.add) {
    get8<G, VEC>(row, v, a.d, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = fma2(f[e], s, r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = mul2(f[e], s);
  }
  put8<G, VEC>(row, v, a.d, r);
}
__device__ __forceinline__ float* part_row(const SumArgs& a, int64_t chunk, int last) {
  return a.part + (2 * chunk + last) * a.ld;
}

constexpr int kAhead = 4;  // rows whose loads are in flight
template <typename T, typename G, bool VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs a) {
  const int group = threadIdx.x / a.width;
  if (group >= a.groups) return;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * a.groups + group;
  const int64_t chunk = item / a.tiles;
  if (chunk >= a.chunks) return;
  const int v = static_cast<int>(item - chunk * a.tiles) * a.width + threadIdx.x - group * a.width;
  if (VEC && 8 * v >= a.d) return;
  pdl_wait();
  const int64_t i0 = chunk * a.len, i1 = min(a.T, i0 + a.len);
  const uint32_t none = static_cast<uint32_t>(a.V);
  uint32_t key = a.keys[i0];
  if (key == none) return;
  // the run that this chunk begins with began before it
  bool open = i0 > 0 && a.keys[i0 - 1] == key;
  f2 sum[4] = {pk(0.f), pk(0.f), pk(0.f), pk(0.f)};
  const T* dout = static_cast<const T*>(a.dout);
  for (int64_t i = i0; i < i1; i += kAhead) {
    Raw8<T> raw[kAhead];
    uint32_t k[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      k[u] = i + u < i1 ? a.keys[i + u] : none;
      if (k[u] != none) load8<VEC>(dout + static_cast<int64_t>(a.tokens[i + u]) * a.d, v, a.d, raw[u]);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (i + u >= i1) break;
      if (k[u] != key) {
        if (open) {
          put8<float, VEC>(part_row(a, chunk, 0), v, a.ld, sum);
        } else {
          put_row<G, VEC>(a, key, v, sum);
        }
        open = false;
        key = k[u];
        if (key == none) return;
        sum[0] = sum[1] = sum[2] = sum[3] = pk(0.f);
      }
      f2 f[4];
      widen(raw[u], f);
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], f[e]);
    }
  }
  if (open) {
    put8<float, VEC>(part_row(a, chunk, 0), v, a.ld, sum);
  } else if (i1 < a.T && a.keys[i1] == key) {
    put8<float, VEC>(part_row(a, chunk, 1), v, a.ld, sum);
  } else {
    put_row<G, VEC>(a, key, v, sum);
  }
}

// Runs that reach over chunk borders.  The chunk that a run begins in adds its own part
// and the first parts of the chunks that follow, up to the one the run ends in.  A warp
// has 256 columns, a block's eight warps every eighth part; then warp 0 adds the eight.
template <typename G, bool VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumArgs a) {
  __shared__ float s_sum[8][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  const int64_t chunk = blockIdx.x;
  const int64_t i0 = chunk * a.len, i1 = i0 + a.len;  // not the last chunk: i1 < T
  const uint32_t key = a.keys[i1 - 1];
  if (key == static_cast<uint32_t>(a.V) || a.keys[i1] != key) return;
  if (i0 > 0 && a.keys[i0] == key && a.keys[i0 - 1] == key) return;  // it began before
  // the last chunk with a part of the run, by bisection over the chunks' first ids
  int64_t lo = chunk + 1, hi = a.chunks - 1;
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) / 2;
    if (a.keys[mid * a.len] == key) lo = mid;
    else hi = mid - 1;
  }
  const int v = blockIdx.y * 32 + lane;
  f2 sum[4] = {pk(0.f), pk(0.f), pk(0.f), pk(0.f)};
  const int64_t parts = lo - chunk + 1;
  for (int64_t q = warp; q < parts; q += 8) {
    f2 f[4];
    get8<float, VEC>(q == 0 ? part_row(a, chunk, 1) : part_row(a, chunk + q, 0), v, a.ld, f);
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], f[e]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = unpk(sum[e]);
    s_sum[warp][64 * e + lane] = x.x;
    s_sum[warp][64 * e + 32 + lane] = x.y;
  }
  __syncthreads();
  if (warp != 0) return;
  const int n = parts < 8 ? static_cast<int>(parts) : 8;
  for (int w = 1; w < n; ++w)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] = add2(sum[e], pk(s_sum[w][64 * e + lane], s_sum[w][64 * e + 32 + lane]));
  put_row<G, VEC>(a, key, v, sum);
}

// ---- sizes -------------------------------------------------------------------
int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Tokens of a chunk: from 8, up to 64 as the batch grows.
int chunk_len(int64_t T) { return T <= 8192 ? 8 : T <= 32768 ? 16 : T <= 131072 ? 32 : 64; }

struct Workspace {
  uint32_t *keys[2], *tokens[2], *counts;
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
  const int64_t len = chunk_len(T), chunks = (T + len - 1) / len;
  q.part = reinterpret_cast<float*>(take(static_cast<size_t>(chunks) * 2 * static_cast<size_t>(round_up(d, 8)) * 4));
  q.bytes = at;
  return q;
}

// ---- launches ----------------------------------------------------------------
template <typename T, typename O>
cudaError_t forward(const moe_embed_desc* q, bool vec, const void* ids, const void* table, void* out, int* status,
                    cudaStream_t s) {
  const int64_t segs = (static_cast<int64_t>(q->d) + 8 * kFwdShares - 1) / (8 * kFwdShares);
  const int64_t blocks = (q->T * segs + kFwdThreads / 32 - 1) / (kFwdThreads / 32);
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(vec ? embed_fwd_kernel<T, O, true> : embed_fwd_kernel<T, O, false>,
                    dim3(static_cast<unsigned>(blocks)), dim3(kFwdThreads), 0, s, ids,
                    q->id_type == MOE_I64 ? 1 : 0, static_cast<const T*>(table), static_cast<int64_t>(q->T), q->V,
                    q->d, q->scale, static_cast<O*>(out), status);
}

cudaError_t zeros(void* p, int64_t bytes, cudaStream_t s) {
  const int64_t to = static_cast<int64_t>(-reinterpret_cast<intptr_t>(p) & 15);
  const int head = static_cast<int>(std::min<int64_t>(to, bytes));
  const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((bytes / 16 + 1023) / 1024, 8 * kSMs));
  return launch_pdl(embed_zero_kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s,
                    static_cast<uint8_t*>(p), bytes, head);
}

// Sorts the tokens by id; the result is in keys[*out], tokens[*out].
cudaError_t sort_tokens(const moe_embed_desc* q, const void* ids, int64_t pad, const Workspace& w, int* status,
                        int* out, cudaStream_t s) {
  const Digits g = digits(q->V);
  const int bins = 1 << g.bits;
  const int64_t n = q->T, chunks = (n + kSortChunk - 1) / kSortChunk;
  Source src = {ids, nullptr, nullptr, q->id_type == MOE_I64 ? 1 : 0, q->V, pad};
  cudaError_t e = cudaSuccess;
  for (int p = 0; p < g.passes && e == cudaSuccess; ++p) {
    const int shift = p * g.bits, to = p & 1;
    e = launch_pdl(sort_count_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kSortThreads), 0, s, src, n, shift,
                   bins, static_cast<int>(chunks), w.counts, p == 0 ? status : nullptr);
    if (e != cudaSuccess) break;
    e = launch_pdl(sort_scan_kernel, dim3(1), dim3(kScanThreads), 0, s, w.counts, chunks * bins);
    if (e != cudaSuccess) break;
    e = launch_pdl(sort_place_kernel, dim3(static_cast<unsigned>(chunks)), dim3(kSortThreads), 0, s, src, n, shift,
                   bins, static_cast<int>(chunks), static_cast<const uint32_t*>(w.counts), w.keys[to], w.tokens[to]);
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
  a.groups = 256 / a.width;
  const int64_t items = a.chunks * a.tiles, blocks = (items + a.groups - 1) / a.groups;
  cudaError_t e = launch_pdl(embed_sum_kernel<T, G, VEC>, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, a);
  if (e != cudaSuccess || a.chunks < 2) return e;
  return launch_pdl(embed_join_kernel<G, VEC>,
                    dim3(static_cast<unsigned>(a.chunks - 1), static_cast<unsigned>((static_cast<int64_t>(a.d) + 255) / 256)),
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
  if (!accumulate) {
    const int64_t bytes = static_cast<int64_t>(desc->V) * desc->d * size_of(desc->table_type);
    e = zeros(dtable, bytes, stream);
  }
  if (any && e == cudaSuccess) {
    const Workspace w = workspace(ws, desc->T, desc->V, desc->d);
    int at = 0;
    e = sort_tokens(desc, ids, pad_id, w, status, &at, stream);
    if (e == cudaSuccess) {
      SumArgs a = {};
      a.dout = dout; a.dtable = dtable; a.keys = w.keys[at]; a.tokens = w.tokens[at]; a.part = w.part;
      a.T = desc->T; a.len = chunk_len(desc->T); a.chunks = (a.T + a.len - 1) / a.len;
      a.V = desc->V; a.d = desc->d; a.ld = static_cast<int>(round_up(desc->d, 8));
      a.scale = desc->scale; a.add = accumulate;
      const bool vec = desc->d % 8 == 0 && !misaligned(dout, 16) && !misaligned(dtable, 16);
      if (desc->row_type == MOE_BF16)
        e = desc->table_type == MOE_BF16 ? sums<bf16_t, bf16_t>(a, vec, stream) : sums<bf16_t, float>(a, vec, stream);
      else
        e = desc->table_type == MOE_BF16 ? sums<float, bf16_t>(a, vec, stream) : sums<float, float>(a, vec, stream);
    }
  }
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
