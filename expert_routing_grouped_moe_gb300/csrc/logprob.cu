// Log probabilities of given tokens, entropy and likeliest tokens of rows of
// logits x, and the gradient of x.  With c = inv_temp log2 e, M a row's largest
// logit, t_e = (x_e - M) c and S = sum 2^t:
//   logp_j = (x_y - M) inv_temp - ln S,   lse = M inv_temp + ln S
//   H = ln S - ln 2 (sum 2^t t) / S
//   dx_e = inv_temp (sum_j g_j (1[e=y_j] - p_e) - gH p_e (ln p_e + H) + gl p_e),  p = 2^t / S
//        = 2^t (A + B t) + inv_temp sum_j g_j 1[e=y_j]
// One pass over a row: a thread keeps the sums relative to a maximum of its own and
// moves them when a logit exceeds it by 2^4 (each logit's t is then off by 4 * 2^-24
// at most, and most words move nothing).  Differences are taken before the factor:
// a row of the type's lowest values, whose product with c would overflow, is then
// uniform as the formula says.
//
// The likeliest n tokens cost the pass over the row one comparison for each word of
// 16 bytes: a thread remembers the largest logit of its words and the word it is
// in.  The n best of a row lie in the words of the n threads whose best is largest
// (were one in another thread, n threads' bests would be above it), so those
// threads' words alone, 1/16 of a long row or less, are read again, and of them
// what reaches the n-th thread's best is sorted.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 4.f;      // how far t may exceed 0 before a thread's sums move
constexpr float kLeast = -1000.f;  // t of a logit of -inf, whose 2^t is 0
constexpr int kMaxTargets = MOE_LOGPROB_MAX_TARGETS, kMaxTop = MOE_LOGPROB_MAX_TOP;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 1024;  // that are sorted at once
constexpr int kWinners = 64;       // threads whose words are read again

struct Args {
  const void* x;
  void* dx;
  int64_t ld, dld;
  int T, V, m, top;
  int t64;               // targets are 64-bit
  int same;              // rows of x and dx have the same alignment
  int64_t ignore;
  float inv_temp, c;
  const void* targets;
  const float *dlogp, *dent, *dlse, *entropy_in;
  const float* stats_in;
  float *logp, *stats, *lse, *entropy, *top_logp;
  int32_t* top_ids;
  int* status;
};

// ---- words of a row -----------------------------------------------------------
// A row is read in words of 16 aligned bytes.  Its first and last may reach past
// it; they are read value by value.  Word i holds values [i E - h, i E - h + E).
template <typename T>
struct Row {
  static constexpr int E = 16 / sizeof(T);
  const T* p;
  int V, h, nw;
  bool head, tail;  // word 0, word nw - 1 are partial (one that is both is the head)
  __device__ __forceinline__ Row(const T* row, int V_) : p(row), V(V_) {
    h = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
    nw = static_cast<int>((static_cast<int64_t>(h) + V + E - 1) / E);
    head = h != 0 || V < E;
    tail = (h + V) % E != 0 && !(nw == 1 && head);
  }
  __device__ __forceinline__ int col(int i) const { return i * E - h; }
  __device__ __forceinline__ uint4 word(int i) const {
    return *reinterpret_cast<const uint4*>(p + static_cast<int64_t>(i) * E - h);
  }
  __device__ __forceinline__ uint4 partial(int i) const;
};
template <>
__device__ __forceinline__ uint4 Row<bf16_t>::partial(int i) const {
  uint32_t w[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int64_t q = static_cast<int64_t>(i) * 8 - h + e;
    w[e] = q >= 0 && q < V ? p[q].bits : 0xFF80u;
  }
  return make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
}
template <>
__device__ __forceinline__ uint4 Row<float>::partial(int i) const {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int64_t q = static_cast<int64_t>(i) * 4 - h + e;
    w[e] = q >= 0 && q < V ? __float_as_uint(p[q]) : 0xFF800000u;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// The pairs of a word, widened; NP of them.
template <typename T>
constexpr int kPairs = 8 / sizeof(T);
__device__ __forceinline__ void pairs(const uint4& q, bf16_t, f2 (&f)[4]) {
  f[0] = pk(bf16lo(q.x), bf16hi(q.x)); f[1] = pk(bf16lo(q.y), bf16hi(q.y));
  f[2] = pk(bf16lo(q.z), bf16hi(q.z)); f[3] = pk(bf16lo(q.w), bf16hi(q.w));
}
__device__ __forceinline__ void pairs(const uint4& q, float, f2 (&f)[2]) {
  f[0] = pk(__uint_as_float(q.x), __uint_as_float(q.y));
  f[1] = pk(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest value of a word (NaN only where there is nothing else).
__device__ __forceinline__ float word_max(const uint4& q, bf16_t) {
  const uint32_t r = max_bf16x2(max_bf16x2(q.x, q.y), max_bf16x2(q.z, q.w));
  return fmaxf(bf16lo(r), bf16hi(r));
}
__device__ __forceinline__ float word_max(const uint4& q, float) {
  return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)),
               fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
}
template <typename T>
__device__ __forceinline__ float word_value(const uint4& q, int e) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if (sizeof(T) == 4) return __uint_as_float(w[e & 3]);
  return __uint_as_float((e & 1) ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
}
__device__ __forceinline__ float value(const bf16_t* p) { return __uint_as_float(uint32_t(p->bits) << 16); }
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ void put(bf16_t* p, float x) { p->bits = static_cast<uint16_t>(pack_bf16x2(x, 0.f)); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 ex2(f2 a) {
  const float2 x = unpk(a);
  return pk(ex2(x.x), ex2(x.y));
}
__device__ __forceinline__ f2 at_least(f2 a, float low) {
  const float2 x = unpk(a);
  return pk(fmaxf(x.x, low), fmaxf(x.y, low));
}

// ---- a thread's sums ------------------------------------------------------------
// S = sum 2^((x - m) c), U = sum 2^t t of the logits seen, relative to m; mx is the
// largest of them.
template <bool ENT>
struct Sums {
  float m = -FLT_MAX, mx = -INFINITY;
  f2 S = pk(0.f), U = pk(0.f);

  template <typename T>
  __device__ __forceinline__ float add(const uint4& q, float c) {
    const float big = word_max(q, T{});
    mx = fmaxf(mx, big);
    if ((big - m) * c > kSlack) move(big, c);
    f2 f[kPairs<T>];
    pairs(q, T{}, f);
    const f2 minus = pk(-m), c2 = pk(c);
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) {
      const f2 t = mul2(add2(f[i], minus), c2), e = ex2(t);
      S = add2(S, e);
      if (ENT) U = fma2(e, at_least(t, kLeast), U);
    }
    return big;
  }
  __device__ __forceinline__ void move(float to, float c) {
    const float by = (m - to) * c, f = ex2(by);
    if (ENT) U = f == 0.f ? pk(0.f) : mul2(fma2(S, pk(by), U), pk(f));
    S = mul2(S, pk(f));
    m = to;
  }
};
// Sums relative to `from` made relative to `to` >= from (both > -inf).
__device__ __forceinline__ void relate(float from, float to, float c, float& S, float& U) {
  const float by = (from - to) * c, f = ex2(by);
  U = f == 0.f ? 0.f : (U + by * S) * f;
  S *= f;
}

// ---- order of tokens --------------------------------------------------------------
// A logit as a whole number of the same order; NaN is 0, the least.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 is +0
  const uint32_t o = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return x == x ? o : 0u;
}
constexpr uint32_t kOrderedInf = 0x007FFFFFu;  // of -inf: no token at or below it is listed
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o & 0x7FFFFFFFu : ~o);
}
// Larger logit first, of equal ones the lower column: as one number, larger first.
__device__ __forceinline__ uint64_t token_key(uint32_t o, uint32_t col) {
  return (static_cast<uint64_t>(o) << 32) | (0xFFFFFFFFu - col);
}

struct TopShared {
  uint64_t cand[kCandidates];
  uint64_t out[kMaxTop];    // the block's n best, in order; 0: none
  uint64_t red[32];
  int win[kWinners];
  int nwin, count;
};

// The n largest of cand[0 .. count), in order, into out (0 past them).
template <int NT>
__device__ __forceinline__ void rank_candidates(TopShared& s, int count, int n) {
  for (int i = threadIdx.x; i < n; i += NT)
    if (i >= count) s.out[i] = 0;
  for (int i = threadIdx.x; i < count; i += NT) {
    const uint64_t key = s.cand[i];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < count; ++j) rank += s.cand[j] > key;
    if (rank < n) s.out[rank] = key;
  }
  __syncthreads();
}

// The n best of words [a, b) of a row, which the block's threads read NT apart, and
// of the partial words edge0 and edge1 (-1: none).  best, best_word: this thread's
// largest logit and the first word that has it.
template <typename T, int NT>
__device__ __forceinline__ void block_top(TopShared& s, const Row<T>& row, int a, int b, int edge0, int edge1,
                                          float best, int best_word, int n) {
  const uint32_t o = best > -INFINITY ? ordered(best) : 0u;
  if (threadIdx.x == 0) s.nwin = s.count = 0;
  uint32_t least = 1;      // the value, and among equal ones the word, of the last thread let in
  int last = 0x7FFFFFFF;
  if (__syncthreads_count(o != 0) > n) {
    uint32_t v = 0;
    int above = NT;
    for (int bit = 31; bit >= 0 && above != n; --bit) {
      const uint32_t trial = v | (1u << bit);
      const int k = __syncthreads_count(o >= trial);
      if (k >= n) v = trial, above = k;
    }
    least = v;
    if (above > kWinners) {  // too many equal ones: those with the first words
      int w = 0;             // the most words that let in fewer than n
      for (int bit = 30; bit >= 0; --bit) {
        const int trial = w | (1 << bit);
        if (__syncthreads_count(o > v || (o == v && best_word < trial)) < n) w = trial;
      }
      last = w;
    }
  }
  if (o != 0 && (o > least || (o == least && best_word <= last))) s.win[atomicAdd(&s.nwin, 1)] = threadIdx.x;
  __syncthreads();
  const int per = (b - a + NT - 1) / NT, items = s.nwin * (per > 0 ? per : 0);
  // every value of these words that may be among the n best, to `take`
  auto scan = [&](auto&& take) {
    for (int it = threadIdx.x; it < items + 2; it += NT) {
      int i;
      uint4 q;
      bool whole = it < items;
      if (whole) {
        const int w = it / per;
        i = a + s.win[w] + (it - w * per) * NT;
        if (i >= b) continue;
        q = row.word(i);
      } else {
        i = it == items ? edge0 : edge1;
        if (i < 0) continue;
        q = row.partial(i);
      }
#pragma unroll
      for (int e = 0; e < Row<T>::E; ++e) {
        const uint32_t v = ordered(word_value<T>(q, e));
        if (v > kOrderedInf && (v > least || (v == least && (!whole || i <= last))))
          take(token_key(v, static_cast<uint32_t>(row.col(i) + e)));
      }
    }
  };
  scan([&](uint64_t key) {
    const int at = atomicAdd(&s.count, 1);
    if (at < kCandidates) s.cand[at] = key;
  });
  __syncthreads();
  const int count = s.count;
  if (count <= kCandidates) {
    rank_candidates<NT>(s, count, n);
    return;
  }
  // more than can be sorted at once: one place after the other
  uint64_t before = ~uint64_t(0);
  for (int r = 0; r < n; ++r) {
    uint64_t top = 0;
    scan([&](uint64_t key) {
      if (key < before && key > top) top = key;
    });
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
      const uint64_t other = __shfl_xor_sync(0xffffffffu, top, i);
      top = other > top ? other : top;
    }
    if ((threadIdx.x & 31) == 0) s.red[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int i = 0; i < NT / 32; ++i) top = s.red[i] > top ? s.red[i] : top;
    if (threadIdx.x == 0) s.out[r] = top;
    before = top;
    __syncthreads();
  }
}

// ---- gradient ----------------------------------------------------------------------
// dx = 2^t (A + B t) of a word, at the word's place in dx.
template <typename T, bool ENT>
__device__ __forceinline__ void gradient_pairs(const uint4& q, float M, float c, float A, float B,
                                               f2 (&f)[kPairs<T>]) {
  pairs(q, T{}, f);
  const f2 minus = pk(-M), c2 = pk(c), a2 = pk(A), b2 = pk(B);
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) {
    const f2 t = mul2(add2(f[i], minus), c2), e = ex2(t);
    f[i] = ENT ? mul2(e, fma2(at_least(t, kLeast), b2, a2)) : mul2(e, a2);
  }
}
__device__ __forceinline__ uint4 narrowed(const f2 (&f)[4], bf16_t) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpk(f[i]);
    w[i] = pack_bf16x2(x.x, x.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ uint4 narrowed(const f2 (&f)[2], float) {
  const float2 x = unpk(f[0]), y = unpk(f[1]);
  return make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
}
// A whole word, or (whole = false, or rows of other alignment) value by value.
template <typename T>
__device__ __forceinline__ void put_word(T* drow, const Row<T>& row, int i, const uint4& w, bool whole) {
  const int64_t at = static_cast<int64_t>(i) * Row<T>::E - row.h;
  if (whole) {
    __stcs(reinterpret_cast<uint4*>(drow + at), w);
    return;
  }
#pragma unroll
  for (int e = 0; e < Row<T>::E; ++e)
    if (at + e >= 0 && at + e < row.V) put(drow + at + e, word_value<T>(w, e));
}
// The gradient of words [a, b), NT apart, and of the partial words edge0 and edge1.
// zero: nothing is read and zeros are written.
template <typename T, int NT, int U, bool ENT>
__device__ __forceinline__ void gradient_words(const Row<T>& row, T* drow, int a, int b, int edge0, int edge1,
                                               bool same, bool zero, float M, float c, float A, float B) {
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  for (int i0 = a + static_cast<int>(threadIdx.x); i0 < b; i0 += NT * U) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q[u] = none;
      if (!zero && i0 + u * NT < b) q[u] = row.word(i0 + u * NT);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * NT >= b) break;
      f2 f[kPairs<T>];
      gradient_pairs<T, ENT>(q[u], M, c, A, B, f);
      put_word<T>(drow, row, i0 + u * NT, zero ? none : narrowed(f, T{}), same);
    }
  }
  if (threadIdx.x < 2) {
    const int i = threadIdx.x == 0 ? edge0 : edge1;
    if (i >= 0) {
      f2 f[kPairs<T>];
      gradient_pairs<T, ENT>(zero ? none : row.partial(i), M, c, A, B, f);
      put_word<T>(drow, row, i, zero ? none : narrowed(f, T{}), false);
    }
  }
}

struct Coefs {
  float A, B;
};
// From the row's sum of dlogp, dentropy, dlse, and S, ln S and ln S - H.
__device__ __forceinline__ Coefs coefs(float sum_g, float dent, float dlse, float S, float log_minus_h,
                                       float inv_temp) {
  const float k = inv_temp / S;
  return {k * (dlse - sum_g + dent * log_minus_h), -k * dent * kLn2};
}

struct Targets {
  int y[kMaxTargets];    // -1: asks for nothing
  float g[kMaxTargets], x[kMaxTargets];
};
// Loads target j of row t; -1 where it is ignored or out of range (then *status).
__device__ __forceinline__ int target(const Args& a, int64_t t, int j, bool tell) {
  const int64_t at = t * a.m + j;
  const int64_t y = a.t64 ? static_cast<const int64_t*>(a.targets)[at]
                          : static_cast<int64_t>(static_cast<const int32_t*>(a.targets)[at]);
  if (y == a.ignore) return -1;
  if (y < 0 || y >= a.V) {
    if (tell) atomicCAS(a.status, 0, kErrBadIds);
    return -1;
  }
  return static_cast<int>(y);
}
// The gradient of target j's logit, where it is the first that names it.
template <typename T>
__device__ __forceinline__ void put_target(const Targets& s, int j, int m, T* drow, float M, float c, float A,
                                           float B, float inv_temp) {
  const int y = s.y[j];
  float g = 0.f;
  for (int i = 0; i < m; ++i)
    if (s.y[i] == y) {
      if (i < j) return;
      g += s.g[i];
    }
  const float t = (s.x[j] - M) * c;
  put(drow + y, fmaf(inv_temp, g, ex2(t) * fmaf(fmaxf(t, kLeast), B, A)));
}

// ---- kernels --------------------------------------------------------------------------
// A cluster of 1 to 8 blocks takes a row, each block a run of its words.  GRAD: the
// gradient follows, from the L2.
template <typename T, int NT, int U, bool TOP, bool ENT, bool GRAD>
__global__ void __launch_bounds__(NT) logprob_kernel(const Args a) {
  __shared__ float s_m[NT / 32], s_S[NT / 32], s_U[NT / 32];
  __shared__ float4 s_part;
  __shared__ Targets s_y;
  __shared__ TopShared s_top;
  const unsigned rank = cluster_ctarank();
  unsigned nc;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nc));
  const int64_t t = blockIdx.x / nc;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + t * a.ld;
  const Row<T> row(x, a.V);
  if (static_cast<int>(threadIdx.x) < a.m) {
    const int y = target(a, t, threadIdx.x, rank == 0);
    s_y.y[threadIdx.x] = y;
    s_y.x[threadIdx.x] = y >= 0 ? value(x + y) : 0.f;
    s_y.g[threadIdx.x] = GRAD && y >= 0 && a.dlogp != nullptr ? a.dlogp[t * a.m + threadIdx.x] : 0.f;
  }
  // this block's whole words, and the partial ones that are its
  const int per = (row.nw + static_cast<int>(nc) - 1) / static_cast<int>(nc);
  const int w0 = min(row.nw, static_cast<int>(rank) * per), w1 = min(row.nw, w0 + per);
  const int first = max(w0, row.head ? 1 : 0), end = min(w1, row.nw - (row.tail ? 1 : 0));
  const int edge0 = row.head && w0 == 0 ? 0 : -1;
  const int edge1 = row.tail && w0 < row.nw && w1 == row.nw ? row.nw - 1 : -1;

  Sums<ENT> sums;
  float best = -INFINITY;
  int best_word = 0;
  for (int i0 = first + static_cast<int>(threadIdx.x); i0 < end; i0 += NT * U) {
    uint4 q[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * NT < end) q[u] = row.word(i0 + u * NT);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (i0 + u * NT >= end) break;
      const float big = sums.template add<T>(q[u], a.c);
      if (TOP && big > best) best = big, best_word = i0 + u * NT;
    }
  }
  if (threadIdx.x < 2) {
    const int i = threadIdx.x == 0 ? edge0 : edge1;
    if (i >= 0) sums.template add<T>(row.partial(i), a.c);
  }

  // over the block
  float M = sums.mx;
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) M = fmaxf(M, s_m[i]);
  M = fmaxf(M, -FLT_MAX);  // nothing but -inf: S stays 0
  float S = sum2(sums.S), Us = ENT ? sum2(sums.U) : 0.f;
  relate(sums.m, M, a.c, S, Us);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, i);
    if (ENT) Us += __shfl_xor_sync(0xffffffffu, Us, i);
  }
  if (lane == 0) s_S[warp] = S, s_U[warp] = Us;
  __syncthreads();
  S = Us = 0.f;
#pragma unroll
  for (int i = 0; i < NT / 32; ++i) S += s_S[i], Us += s_U[i];
  if (TOP) block_top<T, NT>(s_top, row, first, end, edge0, edge1, best, best_word, a.top);

  // over the cluster
  if (nc > 1) {
    if (threadIdx.x == 0) s_part = make_float4(M, S, Us, 0.f);
    cluster_sync();
    float pm[kMaxCluster], ps[kMaxCluster], pu[kMaxCluster];
    const float own = M;
#pragma unroll
    for (unsigned r = 0; r < kMaxCluster; ++r) {
      pm[r] = own, ps[r] = pu[r] = 0.f;
      if (r < nc) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, _}, [%3];"
                     : "=f"(pm[r]), "=f"(ps[r]), "=f"(pu[r])
                     : "r"(mapa_shared(smem_u32(&s_part), r))
                     : "memory");
      }
      M = fmaxf(M, pm[r]);
    }
    S = Us = 0.f;
#pragma unroll
    for (unsigned r = 0; r < kMaxCluster; ++r) {
      relate(pm[r], M, a.c, ps[r], pu[r]);
      S += ps[r];
      Us += pu[r];
    }
    if (TOP && rank == 0) {
      const int total = static_cast<int>(nc) * a.top;
      for (int i = threadIdx.x; i < total; i += NT) {
        uint64_t key;
        const unsigned r = static_cast<unsigned>(i / a.top);
        asm volatile("ld.shared::cluster.u64 %0, [%1];"
                     : "=l"(key)
                     : "r"(mapa_shared(smem_u32(&s_top.out[i - r * a.top]), r))
                     : "memory");
        s_top.cand[i] = key;
      }
      __syncthreads();  // s_top.out of this block was read above, before it is written
      // empty places (0) of several blocks are equal: they rank past every token
      const uint64_t key = static_cast<int>(threadIdx.x) < total ? s_top.cand[threadIdx.x] : 0;
      static_assert(kMaxCluster * kMaxTop <= 256, "a thread for each key, or two");
      for (int i = threadIdx.x; i < a.top; i += NT) s_top.out[i] = 0;
      __syncthreads();
      for (int i = threadIdx.x; i < total; i += NT) {
        const uint64_t k = i == static_cast<int>(threadIdx.x) ? key : s_top.cand[i];
        int place = 0;
        for (int j = 0; j < total; ++j) place += s_top.cand[j] > k;
        if (k != 0 && place < a.top) s_top.out[place] = k;
      }
      __syncthreads();
    }
  }

  const bool empty = S == 0.f;
  const float log_S = logf(S);
  if (rank == 0) {
    if (static_cast<int>(threadIdx.x) < a.m)
      a.logp[t * a.m + threadIdx.x] =
          s_y.y[threadIdx.x] < 0 ? 0.f : empty ? -INFINITY : (s_y.x[threadIdx.x] - M) * a.inv_temp - log_S;
    if (threadIdx.x == 0) {
      a.stats[2 * t] = M;
      a.stats[2 * t + 1] = S;
      if (a.lse != nullptr) a.lse[t] = empty ? -INFINITY : fmaf(M, a.inv_temp, log_S);
      if (ENT && a.entropy != nullptr) a.entropy[t] = empty ? 0.f : log_S - kLn2 * Us / S;
    }
    if (TOP && static_cast<int>(threadIdx.x) < a.top) {
      const uint64_t key = s_top.out[threadIdx.x];
      const int64_t at = t * a.top + threadIdx.x;
      if (a.top_ids != nullptr) a.top_ids[at] = key != 0 ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
      if (a.top_logp != nullptr)
        a.top_logp[at] = key != 0 ? (from_ordered(static_cast<uint32_t>(key >> 32)) - M) * a.inv_temp - log_S : -INFINITY;
    }
  }
  if (GRAD) {
    float sum_g = 0.f;
    bool some = false;
    for (int j = 0; j < a.m; ++j) {
      sum_g += s_y.g[j];
      some |= s_y.g[j] != 0.f;
    }
    const float dent = ENT && a.dent != nullptr ? a.dent[t] : 0.f, dlse = a.dlse != nullptr ? a.dlse[t] : 0.f;
    const bool zero = empty || !(some || dent != 0.f || dlse != 0.f);
    const Coefs k = coefs(sum_g, dent, dlse, S, ENT ? kLn2 * Us / S : 0.f, a.inv_temp);
    T* drow = static_cast<T*>(a.dx) + t * a.dld;
    gradient_words<T, NT, U, ENT>(row, drow, first, end, edge0, edge1, a.same != 0, zero, M, a.c, k.A, k.B);
    __syncthreads();
    if (!zero && static_cast<int>(threadIdx.x) < a.m && s_y.y[threadIdx.x] >= 0) {
      const int w = (s_y.y[threadIdx.x] + row.h) / Row<T>::E;
      if (w >= w0 && w < w1) put_target<T>(s_y, threadIdx.x, a.m, drow, M, a.c, k.A, k.B, a.inv_temp);
    }
  }
  if (nc > 1) cluster_sync();  // no block leaves while its shared memory is read
}

// The gradient alone: units of kBwdThreads * kBwdWords words of a row.
constexpr int kBwdThreads = 256, kBwdWords = 4, kBwdUnit = kBwdThreads * kBwdWords;
template <typename T, bool ENT>
__global__ void __launch_bounds__(kBwdThreads) logprob_bwd_kernel(const Args a, int chunks, int64_t units) {
  __shared__ Targets s_y;
  const int lane = threadIdx.x & 31;
  pdl_wait();
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t t = unit / chunks;
    const int chunk = static_cast<int>(unit - t * chunks);
    const T* x = static_cast<const T*>(a.x) + t * a.ld;
    const Row<T> row(x, a.V);
    const int w0 = chunk * kBwdUnit, w1 = min(row.nw, w0 + kBwdUnit);
    if (w0 >= w1) continue;
    const int first = max(w0, row.head ? 1 : 0), end = min(w1, row.nw - (row.tail ? 1 : 0));
    const int edge0 = row.head && w0 == 0 ? 0 : -1, edge1 = row.tail && w1 == row.nw ? row.nw - 1 : -1;
    float sum_g = 0.f;
    bool some = false, here = false;
    for (int j0 = 0; j0 < a.m; j0 += 32) {
      int y = -1;
      float g = 0.f;
      if (j0 + lane < a.m) {
        y = target(a, t, j0 + lane, false);
        if (y >= 0 && a.dlogp != nullptr) g = a.dlogp[t * a.m + j0 + lane];
      }
      some |= __any_sync(0xffffffffu, g != 0.f);
      const int w = (y + row.h) / Row<T>::E;
      here |= __any_sync(0xffffffffu, y >= 0 && w >= w0 && w < w1);
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) g += __shfl_xor_sync(0xffffffffu, g, i);
      sum_g += g;
    }
    const float M = a.stats_in[2 * t], S = a.stats_in[2 * t + 1];
    const float dent = ENT ? a.dent[t] : 0.f, dlse = a.dlse != nullptr ? a.dlse[t] : 0.f;
    const bool zero = S == 0.f || !(some || dent != 0.f || dlse != 0.f);
    const Coefs k = coefs(sum_g, dent, dlse, S, ENT ? logf(S) - a.entropy_in[t] : 0.f, a.inv_temp);
    here &= !zero;  // the same for every warp
    int mine = -1;
    if (here) {
      // targets' logits are read before any word of theirs is overwritten
      if (static_cast<int>(threadIdx.x) < a.m) {
        const int y = target(a, t, threadIdx.x, false);
        s_y.y[threadIdx.x] = y;
        s_y.g[threadIdx.x] = y >= 0 && a.dlogp != nullptr ? a.dlogp[t * a.m + threadIdx.x] : 0.f;
        const int w = (y + row.h) / Row<T>::E;
        if (y >= 0 && w >= w0 && w < w1) mine = y;
        s_y.x[threadIdx.x] = mine >= 0 ? value(x + y) : 0.f;
      }
      __syncthreads();
    }
    T* drow = static_cast<T*>(a.dx) + t * a.dld;
    gradient_words<T, kBwdThreads, kBwdWords, ENT>(row, drow, first, end, edge0, edge1, a.same != 0, zero, M,
                                                   a.c, k.A, k.B);
    if (here) {
      __syncthreads();
      if (mine >= 0) put_target<T>(s_y, threadIdx.x, a.m, drow, M, a.c, k.A, k.B, a.inv_temp);
      __syncthreads();  // before s_y is written again
    }
  }
}

// ---- launches -----------------------------------------------------------------------------
// Threads of a block: 128 for rows of up to 2048 words, else 512.  Blocks of a row:
// one where there are two rows for each SM, more where there are fewer; always eight
// for the step, so that the rows in flight (about 80) stay in the L2 until their
// second reading.
constexpr int kShortWords = 2048;

template <typename T, int NT, bool TOP, bool ENT, bool GRAD>
cudaError_t row_kernel(const Args& a, unsigned cluster, cudaStream_t s) {
  return launch_pdl_cluster(logprob_kernel<T, NT, 4, TOP, ENT, GRAD>,
                            dim3(static_cast<unsigned>(a.T) * cluster), dim3(NT), 0, s, cluster, a);
}
template <typename T, int NT>
cudaError_t rows(const Args& a, bool grad, unsigned cluster, cudaStream_t s) {
  const bool ent = a.entropy != nullptr || a.dent != nullptr, top = a.top > 0;
  if (grad)
    return top ? (ent ? row_kernel<T, NT, true, true, true>(a, cluster, s)
                      : row_kernel<T, NT, true, false, true>(a, cluster, s))
               : (ent ? row_kernel<T, NT, false, true, true>(a, cluster, s)
                      : row_kernel<T, NT, false, false, true>(a, cluster, s));
  return top ? (ent ? row_kernel<T, NT, true, true, false>(a, cluster, s)
                    : row_kernel<T, NT, true, false, false>(a, cluster, s))
             : (ent ? row_kernel<T, NT, false, true, false>(a, cluster, s)
                    : row_kernel<T, NT, false, false, false>(a, cluster, s));
}
template <typename T>
cudaError_t launch_rows(const Args& a, bool grad, cudaStream_t s) {
  const int words = static_cast<int>((static_cast<int64_t>(a.V) * sizeof(T) + 15) / 16);
  if (words <= kShortWords) return rows<T, 128>(a, grad, 1, s);
  unsigned cluster = kMaxCluster;
  if (!grad)
    while (cluster > 1 && static_cast<int64_t>(a.T) * cluster >= 4 * kSMs) cluster /= 2;
  return rows<T, 512>(a, grad, cluster, s);
}
template <typename T>
cudaError_t launch_bwd(const Args& a, cudaStream_t s) {
  constexpr int E = Row<T>::E;
  const int64_t words = (static_cast<int64_t>(a.V) + 2 * E - 2) / E;
  const int64_t chunks = (words + kBwdUnit - 1) / kBwdUnit, units = chunks * a.T;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(units, 0x7FFFFFFF));
  return launch_pdl(a.dent != nullptr ? logprob_bwd_kernel<T, true> : logprob_bwd_kernel<T, false>, dim3(grid),
                    dim3(kBwdThreads), 0, s, a, static_cast<int>(chunks), units);
}

int bad(const char* msg) { return record_error(MOE_ERR_INVALID_ARG, msg); }
bool misaligned(const void* p, unsigned size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; }

int check_desc(const moe_logprob_desc* q, bool grad) {
  if (q == nullptr) return bad("desc is NULL");
  if (q->T < 0 || q->V <= 0) return bad("T must not be negative, V must be positive");
  if (q->V > 0x7FFFFF00) return record_error(MOE_ERR_UNSUPPORTED, "V is too large");
  if (q->type != MOE_F32 && q->type != MOE_BF16) return bad("type must be MOE_F32 or MOE_BF16");
  if (q->target_type != MOE_I32 && q->target_type != MOE_I64) return bad("target_type must be MOE_I32 or MOE_I64");
  if (q->m < 1 || q->m > kMaxTargets) return bad("m must be in 1 .. MOE_LOGPROB_MAX_TARGETS");
  if (q->top < 0 || q->top > kMaxTop) return bad("top must be in 0 .. MOE_LOGPROB_MAX_TOP");
  if (q->T > 1 && (q->ld < q->V || (grad && q->dld < q->V))) return bad("a row stride is below V");
  if (!(q->inv_temp > 0.f) || !std::isfinite(q->inv_temp)) return bad("inv_temp must be positive");
  if (static_cast<int64_t>(q->T) * kMaxCluster > 0x7FFFFFFF) return record_error(MOE_ERR_UNSUPPORTED, "T is too large");
  return MOE_OK;
}

// What forward and backward share.
int fill(const moe_logprob_desc* q, const void* logits, const void* targets, Args& a) {
  if (!logits || !targets) return bad("logits or targets is NULL");
  if (misaligned(logits, q->type == MOE_BF16 ? 2 : 4)) return bad("logits is misaligned");
  if (misaligned(targets, q->target_type == MOE_I64 ? 8 : 4)) return bad("targets is misaligned");
  a.x = logits; a.targets = targets;
  a.ld = q->ld; a.dld = q->dld; a.T = q->T; a.V = q->V; a.m = q->m; a.top = q->top;
  a.t64 = q->target_type == MOE_I64; a.ignore = q->ignore_id;
  a.inv_temp = q->inv_temp;
  a.c = static_cast<float>(static_cast<double>(q->inv_temp) * 1.4426950408889634074);
  return MOE_OK;
}
int fill_grad(const moe_logprob_desc* q, const float* dlogp, const float* dent, const float* dlse,
              void* dlogits, Args& a) {
  if (!dlogits) return bad("dlogits is NULL");
  if (misaligned(dlogits, q->type == MOE_BF16 ? 2 : 4)) return bad("dlogits is misaligned");
  if (misaligned(dlogp, 4) || misaligned(dent, 4) || misaligned(dlse, 4)) return bad("misaligned gradient");
  if (dlogits == a.x && q->T > 1 && q->dld != q->ld) return bad("dlogits in the place of logits needs their row stride");
  a.dx = dlogits; a.dlogp = dlogp; a.dent = dent; a.dlse = dlse;
  const uintptr_t size = q->type == MOE_BF16 ? 2 : 4;
  a.same = ((reinterpret_cast<uintptr_t>(dlogits) - reinterpret_cast<uintptr_t>(a.x)) & 15u) == 0 &&
           (q->T == 1 || ((static_cast<uintptr_t>(q->dld - q->ld) * size) & 15u) == 0);
  return MOE_OK;
}
int fill_out(const moe_logprob_desc* q, float* logp, float* stats, float* lse, float* entropy,
             int32_t* top_ids, float* top_logp, Args& a) {
  if (!logp || !stats) return bad("logp or stats is NULL");
  if (misaligned(logp, 4) || misaligned(stats, 4) || misaligned(lse, 4) || misaligned(entropy, 4) ||
      misaligned(top_ids, 4) || misaligned(top_logp, 4))
    return bad("misaligned output");
  if (q->top == 0 && (top_ids || top_logp)) return bad("top_ids and top_logp go with top > 0");
  a.logp = logp; a.stats = stats; a.lse = lse; a.entropy = entropy; a.top_ids = top_ids; a.top_logp = top_logp;
  if (!top_ids && !top_logp) a.top = 0;
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_logprob_fwd(const moe_logprob_desc* desc, const void* logits, const void* targets, float* logp,
                    float* stats, float* lse, float* entropy, int32_t* top_ids, float* top_logp,
                    moe_stream_t stream) {
  NvtxScope nvtx("moe_logprob_fwd");
  int rc = check_desc(desc, false);
  if (rc) return rc;
  if (desc->T == 0) return record_error(MOE_OK, "");
  Args a = {};
  if ((rc = fill(desc, logits, targets, a)) || (rc = fill_out(desc, logp, stats, lse, entropy, top_ids, top_logp, a)) || (rc = device_status_word(&a.status)))
    return rc;
  ProbeScope probe("logprob_fwd", stream);
  const cudaError_t e = desc->type == MOE_BF16 ? launch_rows<bf16_t>(a, false, stream)
                                               : launch_rows<float>(a, false, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

int moe_logprob_bwd(const moe_logprob_desc* desc, const void* logits, const void* targets,
                    const float* stats, const float* entropy, const float* dlogp, const float* dentropy,
                    const float* dlse, void* dlogits, moe_stream_t stream) {
  NvtxScope nvtx("moe_logprob_bwd");
  int rc = check_desc(desc, true);
  if (rc) return rc;
  if (desc->T == 0) return record_error(MOE_OK, "");
  Args a = {};
  if ((rc = fill(desc, logits, targets, a)) || (rc = fill_grad(desc, dlogp, dentropy, dlse, dlogits, a))) return rc;
  if (!stats || misaligned(stats, 4)) return bad("stats NULL or misaligned");
  if (dentropy && (!entropy || misaligned(entropy, 4))) return bad("dentropy needs entropy");
  a.stats_in = stats; a.entropy_in = entropy;
  ProbeScope probe("logprob_bwd", stream);
  const cudaError_t e = desc->type == MOE_BF16 ? launch_bwd<bf16_t>(a, stream) : launch_bwd<float>(a, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

int moe_logprob_step(const moe_logprob_desc* desc, const void* logits, const void* targets,
                     const float* dlogp, const float* dentropy, const float* dlse, float* logp,
                     float* stats, float* lse, float* entropy, int32_t* top_ids, float* top_logp,
                     void* dlogits, moe_stream_t stream) {
  NvtxScope nvtx("moe_logprob_step");
  int rc = check_desc(desc, true);
  if (rc) return rc;
  if (desc->T == 0) return record_error(MOE_OK, "");
  Args a = {};
  if ((rc = fill(desc, logits, targets, a)) || (rc = fill_grad(desc, dlogp, dentropy, dlse, dlogits, a)) ||
      (rc = fill_out(desc, logp, stats, lse, entropy, top_ids, top_logp, a)) || (rc = device_status_word(&a.status)))
    return rc;
  ProbeScope probe("logprob_step", stream);
  const cudaError_t e = desc->type == MOE_BF16 ? launch_rows<bf16_t>(a, true, stream)
                                               : launch_rows<float>(a, true, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
