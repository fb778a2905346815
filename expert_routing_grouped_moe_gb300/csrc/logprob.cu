// Log probabilities of given tokens, entropy and likeliest tokens of rows of
// logits x, and the gradient of x.  With c = inv_temp log2 e, M a row's largest
// logit, t_e = (x_e - M) c and S = sum 2^t:
//   logp_j = (x_y - M) inv_temp - ln S,   lse = M inv_temp + ln S
//   H = ln S - ln 2 (sum 2^t t) / S
//   dx_e = inv_temp (sum_j g_j (1[e=y_j] - p_e) - gH p_e (ln p_e + H) + gl p_e),  p = 2^t / S
//        = 2^t (A + B t) + inv_temp sum_j g_j 1[e=y_j]
// One pass over a row: a thread keeps the sums relative to a shift of its own, t = x c -
// shift in one fused operation, and moves them when a logit exceeds it by 2^4 (each t
// is then off by 4 * 2^-24 at most, and most words move nothing).  The row's shift is
// its largest logit times c, rounded, the same for every use.  That rounding is half a
// step of M c, so it takes rows with |M c| below 2^22; the others (all of a row masked
// by some low value, say) are summed once more with t = (x - M) c.  Lower logits than
// that are no shift of a thread's either: next to such a row's largest they are nothing.
//
// The likeliest n tokens cost the pass over the row next to nothing: a thread has the
// largest logit of its words at hand, and notes it for each quarter of them.  The n best
// of a row lie in the n such parts with the largest best (were one in another part, n
// parts' bests would be above it), so those parts' words alone, 1/50 of a long row for
// 20 tokens, are read again, and of them what reaches the n-th part's best is sorted.
//
// Memory bounds all of it.  4096 rows of 151936 bf16 logits, of a copy's rate: forward
// 187 us (0.98), with entropy 196, with 20 tokens listed 220; backward 357 (1.03); both
// in one call 425 to 438 (0.86, 0.84), whose second reading misses the L2 now and then.  One row: 8.5
// us, a chain of short steps.  Rows a little above the number of blocks that run at once
// take two turns: 1500 of 151936 run at 0.92, 1250 at 0.85.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kSlack = 4.f;      // how far t may exceed 0 before a thread's sums move
constexpr float kLeast = -1000.f;  // t of a logit of -inf, whose 2^t is 0
// |M c| from which a row is extreme (the rounding of M c is 2^-3 at most below it); a
// thread's shift before it saw a logit above that, below every other row's; and what x c
// counts as where t is needed and x c is lower still.  Apart by 2^21 each, so that 2^t is 0
// from one to the next, and small enough for t times any gradient to stay finite.
constexpr float kExtreme = 0x1p22f, kUnset = -0x1.8p22f, kFloor = -0x1p23f;
constexpr int kMaxTargets = MOE_LOGPROB_MAX_TARGETS, kMaxTop = MOE_LOGPROB_MAX_TOP;
constexpr int kMaxCluster = 8;
constexpr int kCandidates = 512;   // that are sorted at once
constexpr int kWinners = 64;       // parts whose words are read again

struct Args {
  const void* x;
  void* dx;
  int64_t ld, dld;
  int T, V, m, top;
  int t64;               // targets are 64-bit
  int same;              // rows of x and dx have the same alignment
  int64_t ignore;
  float inv_temp, c;
  uint32_t floor;        // kFloor / c: as fp32, or twice as bf16
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
  __device__ __forceinline__ const uint4* at(int i) const {
    return reinterpret_cast<const uint4*>(p + static_cast<int64_t>(i) * E - h);
  }
  __device__ __forceinline__ uint4 word(int i) const { return *at(i); }
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
// The word with values of at least `low` (NaN stays).
__device__ __forceinline__ uint4 at_least(uint4 q, uint32_t low, bf16_t) {
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(q.x) : "r"(low));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(q.y) : "r"(low));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(q.z) : "r"(low));
  asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(q.w) : "r"(low));
  return q;
}
__device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  return __float_as_uint(r);
}
__device__ __forceinline__ uint4 at_least(const uint4& q, uint32_t low, float) {
  return make_uint4(max_nan(q.x, low), max_nan(q.y, low), max_nan(q.z, low), max_nan(q.w, low));
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

// ---- a thread's sums ------------------------------------------------------------
// S = sum 2^t and U = sum 2^t t of the logits seen, t = x c - at; mx: the largest logit.
template <bool ENT>
struct Sums {
  float at = kUnset, mx = -INFINITY;
  f2 S = pk(0.f), U = pk(0.f);

  template <typename T>
  __device__ __forceinline__ void add(uint4 q, float c, uint32_t floor) {
    const float big = word_max(q, T{});
    mx = fmaxf(mx, big);
    if (fmaf(big, c, -at) > kSlack) move(big * c);
    if (ENT) q = at_least(q, floor, T{});
    f2 f[kPairs<T>];
    pairs(q, T{}, f);
    const f2 minus = pk(-at), c2 = pk(c);
#pragma unroll
    for (int i = 0; i < kPairs<T>; ++i) {
      const f2 t = fma2(f[i], c2, minus), e = ex2(t);
      S = add2(S, e);
      if (ENT) U = fma2(e, t, U);
    }
  }
  __device__ __forceinline__ void move(float to) {
    const float by = at - to, f = ex2(by);
    if (ENT) U = f == 0.f ? pk(0.f) : mul2(fma2(S, pk(by), U), pk(f));
    S = mul2(S, pk(f));
    at = to;
  }
};
// Sums relative to `from` made relative to `to` >= from.
__device__ __forceinline__ void relate(float from, float to, float& S, float& U) {
  const float by = from - to, f = ex2(by);
  U = f == 0.f ? 0.f : (U + by * S) * f;
  S *= f;
}
// What a row's exponents are taken relative to.
struct Shift {
  float M, at, c;
  bool extreme;
  __device__ __forceinline__ Shift(float M_, float c_) : M(M_), at(M_ * c_), c(c_) {
    extreme = !(fabsf(at) < kExtreme);
  }
  __device__ __forceinline__ float t(float x) const { return extreme ? (x - M) * c : fmaf(x, c, -at); }
  // ln of x's share of a sum.  Where t overflows, its factor log2 e may be all that did.
  __device__ __forceinline__ float log_share(float x, float log_S, float inv_temp) const {
    const float e = t(x);
    return e == -INFINITY ? (x - M) * inv_temp - log_S : fmaf(kLn2, e, -log_S);
  }
};
// An extreme row's sums, its largest logit known.
template <typename T>
__device__ __forceinline__ void add_extreme(const uint4& q, const Shift& h, float& S, float& U) {
#pragma unroll
  for (int e = 0; e < 16 / static_cast<int>(sizeof(T)); ++e) {
    const float t = (word_value<T>(q, e) - h.M) * h.c, p = ex2(t);
    S += p;
    U += p * fmaxf(t, kLeast);
  }
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

constexpr int kBuckets = 64;
struct TopShared {
  int bucket[kBuckets];
  uint64_t cand[kCandidates];
  uint64_t out[kMaxTop];    // the block's n best, in order; 0: none
  uint64_t red[32];
  int win[kWinners];        // first word, from the block's first on, of a part that is read again
  int nwin, count, above;
  uint32_t least;
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

// A thread's words are seen in P parts, each a run of `step` words of the block's (a
// multiple of NT; the last may be shorter): the largest logit of a part stands for it.
// Four in blocks of 256 threads, whose threads have up to 75 words of a row of 151936
// logits, one in others.
template <int NT>
constexpr int kParts = NT == 256 ? 4 : 1;

// The n best of words [a, b) of a row, which the block's threads read NT apart, and of
// the partial words edge0 and edge1 (-1: none).  s_best: the order of the largest
// logit of each part of each thread; largest: of all of them, or above.
template <typename T, int NT>
__device__ __forceinline__ void block_top(TopShared& s, uint32_t (&s_best)[kParts<NT> * NT], const Row<T>& row, int a,
                                          int b, int step, int edge0, int edge1, uint32_t largest, int n) {
  constexpr int P = kParts<NT>;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) s.nwin = s.count = 0;
  for (int i = threadIdx.x; i < kBuckets; i += NT) s.bucket[i] = 0;
  __syncthreads();
  // What the parts' orders have to reach: first from counts of them in buckets of four steps
  // of a bf16 below the largest, which let in a few more than n.
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t o = s_best[i * NT + threadIdx.x], below = (largest >> 16) - (o >> 16);
    if (o != 0 && below / 4 < kBuckets) atomicAdd(&s.bucket[below / 4], 1);
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int b0 = s.bucket[2 * lane], b1 = s.bucket[2 * lane + 1];
    int upto = b0 + b1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int q = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += q;
    }
    const unsigned enough = __ballot_sync(0xffffffffu, upto >= n);
    uint32_t v = 1;
    int above = -1;
    if (enough != 0) {
      const int l = __ffs(enough) - 1;
      const int all = __shfl_sync(0xffffffffu, upto, l), less = __shfl_sync(0xffffffffu, upto - b1, l);
      above = less >= n ? less : all;
      const uint32_t reach = 4 * (2 * l + (less >= n ? 0 : 1)) + 3, top = largest >> 16;
      v = max(1u, (top > reach ? top - reach : 0u) << 16);
    }
    // where the n are further down, or too many that near: the largest v that n of them
    // reach, bit by bit
    if (above < 0 || above > kWinners) {
      constexpr int kFew = P * NT / 32;  // parts that a lane looks at
      uint32_t o[kFew];
      above = 0;
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        o[i] = s_best[32 * i + lane];
        above += o[i] != 0;
      }
      above = __reduce_add_sync(0xffffffffu, above);
      v = 1;
      if (above > n) {
        v = 0;
        for (int bit = 31; bit >= (sizeof(T) == 2 ? 16 : 0) && above != n; --bit) {  // bf16: 16 bits
          int k = 0;
#pragma unroll
          for (int i = 0; i < kFew; ++i) k += o[i] >= (v | (1u << bit));
          k = __reduce_add_sync(0xffffffffu, k);
          if (k >= n) v |= 1u << bit, above = k;
        }
        // the last 16 bits of a bf16's order are its sign's: ones where it is negative
        if (sizeof(T) == 2 && !(v & 0x80000000u)) v |= 0xFFFFu;
      }
    }
    if (lane == 0) s.least = v, s.above = above;
  }
  __syncthreads();
  const uint32_t least = s.least;
  int last = 0x7FFFFFFF;
  int best_word[P];
  if (s.above > kWinners) {  // too many equal ones: those whose first such word comes first
#pragma unroll
    for (int i = 0; i < P; ++i) {
      best_word[i] = 0;
      if (s_best[i * NT + threadIdx.x] == least) {
        const int to = min(b, a + (i + 1) * step);
        for (best_word[i] = a + i * step + static_cast<int>(threadIdx.x); best_word[i] < to; best_word[i] += NT)
          if (ordered(word_max(row.word(best_word[i]), T{})) == least) break;
      }
    }
    int w = 0;  // the most words that let in fewer than n
    for (int bit = 30; bit >= 0; --bit) {
      const int trial = w | (1 << bit);
      int k = 0;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint32_t o = s_best[i * NT + threadIdx.x];
        k += o > least || (o == least && best_word[i] < trial);
      }
      k = __reduce_add_sync(0xffffffffu, k);
      if (lane == 0) s.red[threadIdx.x >> 5] = k;
      __syncthreads();
      int all = 0;
      for (int i = 0; i < NT / 32; ++i) all += static_cast<int>(s.red[i]);
      if (all < n) w = trial;
      __syncthreads();
    }
    last = w;
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const uint32_t o = s_best[i * NT + threadIdx.x];
    if (o != 0 && (o > least || (o == least && (last == 0x7FFFFFFF || best_word[i] <= last)))) {
      const int at = atomicAdd(&s.nwin, 1);  // n at most, or kWinners
      if (at < kWinners) s.win[at] = i * step + threadIdx.x;
    }
  }
  __syncthreads();
  const int per = step / NT, items = min(s.nwin, kWinners) * per;
  // every value of these words that may be among the n best, to `take`; a few words' loads
  // at once (a long row's words may have left the L2)
  auto scan = [&](auto&& take) {
    auto values = [&](const uint4& q, int i, int to) {
      if (ordered(word_max(q, T{})) < least) return;
#pragma unroll
      for (int e = 0; e < Row<T>::E; ++e) {
        const uint32_t v = ordered(word_value<T>(q, e));
        if (v > kOrderedInf && (v > least || (v == least && i <= to)))
          take(token_key(v, static_cast<uint32_t>(row.col(i) + e)));
      }
    };
    constexpr int B = 3;
    for (int it = threadIdx.x; it < items; it += B * NT) {
      uint4 q[B];
      int at[B];
#pragma unroll
      for (int u = 0; u < B; ++u) {
        at[u] = b;
        if (it + u * NT < items) {
          const int w = (it + u * NT) / per, first = s.win[w];
          at[u] = a + first + (it + u * NT - w * per) * NT;
        }
        if (at[u] < b) q[u] = row.word(at[u]);
      }
#pragma unroll
      for (int u = 0; u < B; ++u)
        if (at[u] < b) values(q[u], at[u], last);
    }
    if (threadIdx.x < 2) {
      const int i = threadIdx.x == 0 ? edge0 : edge1;
      if (i >= 0) values(row.partial(i), i, 0x7FFFFFFF);
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
    if (lane == 0) s.red[threadIdx.x >> 5] = top;
    __syncthreads();
    for (int i = 0; i < NT / 32; ++i) top = s.red[i] > top ? s.red[i] : top;
    if (threadIdx.x == 0) s.out[r] = top;
    before = top;
    __syncthreads();
  }
}

// ---- gradient ----------------------------------------------------------------------
// dx = 2^t (A + B t) of a word.
template <typename T, bool ENT, bool EXTREME>
__device__ __forceinline__ void gradient_pairs(uint4 q, const Shift& h, uint32_t floor, float A, float B,
                                               f2 (&f)[kPairs<T>]) {
  if (ENT && !EXTREME) q = at_least(q, floor, T{});
  pairs(q, T{}, f);
  const f2 minus = pk(EXTREME ? -h.M : -h.at), c2 = pk(h.c), a2 = pk(A), b2 = pk(B);
#pragma unroll
  for (int i = 0; i < kPairs<T>; ++i) {
    f2 t;
    if (EXTREME) {
      const float2 x = unpk(mul2(add2(f[i], minus), c2));
      t = pk(fmaxf(x.x, kLeast), fmaxf(x.y, kLeast));
    } else {
      t = fma2(f[i], c2, minus);
    }
    const f2 e = ex2(t);
    f[i] = ENT ? mul2(e, fma2(t, b2, a2)) : mul2(e, a2);
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
template <typename T>
__device__ __forceinline__ void put_values(T* drow, const Row<T>& row, int i, const uint4& w) {
  const int64_t at = static_cast<int64_t>(i) * Row<T>::E - row.h;
#pragma unroll
  for (int e = 0; e < Row<T>::E; ++e)
    if (at + e >= 0 && at + e < row.V) put(drow + at + e, word_value<T>(w, e));
}
// The gradient of words [a, b), NT apart from thread `id` on, and of the partial words
// edge0 and edge1; words come from word(i).  zero: nothing is read, zeros are written.
// same: rows of dx have the alignment of x's, so that whole words are written.
template <typename T, int NT, int U, bool ENT, typename Word>
__device__ __forceinline__ void gradient_words(const Row<T>& row, T* drow, int id, int a, int b, int edge0,
                                               int edge1, bool same, bool zero, const Shift& h, uint32_t floor,
                                               float A, float B, Word&& word) {
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  auto slow = [&](const uint4& q) {
    f2 f[kPairs<T>];
    if (h.extreme) gradient_pairs<T, ENT, true>(q, h, floor, A, B, f);
    else gradient_pairs<T, ENT, false>(q, h, floor, A, B, f);
    return narrowed(f, T{});
  };
  uint4* to = reinterpret_cast<uint4*>(drow - row.h);
  if (zero && same) {
    for (int i = a + id; i < b; i += NT) __stcs(to + i, none);
  } else if (same && !h.extreme) {
    int i = a + id;
    for (; i + (U - 1) * NT < b; i += NT * U) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = word(i + u * NT);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f2 f[kPairs<T>];
        gradient_pairs<T, ENT, false>(q[u], h, floor, A, B, f);
        __stcs(to + i + u * NT, narrowed(f, T{}));
      }
    }
#pragma unroll 1
    for (; i < b; i += NT) {
      f2 f[kPairs<T>];
      gradient_pairs<T, ENT, false>(word(i), h, floor, A, B, f);
      __stcs(to + i, narrowed(f, T{}));
    }
  } else {
#pragma unroll 1
    for (int i = a + id; i < b; i += NT) {
      const uint4 w = zero ? none : slow(word(i));
      if (same) __stcs(to + i, w);
      else put_values(drow, row, i, w);
    }
  }
  if (id < 2) {
    const int i = id == 0 ? edge0 : edge1;
    if (i >= 0) put_values(drow, row, i, zero ? none : slow(row.partial(i)));
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
// The gradient of target j's logit: the first that names a token adds up what all get.
template <typename T>
__device__ __forceinline__ void put_target(const Targets& s, int j, int m, T* drow, const Shift& h, float A,
                                           float B, float inv_temp) {
  const int y = s.y[j];
  float g = 0.f;
  for (int i = 0; i < m; ++i)
    if (s.y[i] == y) {
      if (i < j) return;
      g += s.g[i];
    }
  const float t = h.t(s.x[j]);
  put(drow + y, fmaf(inv_temp, g, ex2(t) * fmaf(fmaxf(t, kLeast), B, A)));
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ---- kernels --------------------------------------------------------------------------
// A cluster of 1 to 8 blocks takes a row, each block a run of its words.  GRAD: the
// gradient follows, from a second reading that the L2 serves.
template <typename T, int NT, int MINB, int U, bool TOP, bool ENT, bool GRAD>
__global__ void __launch_bounds__(NT, MINB) logprob_kernel(const Args a) {
  constexpr int W = NT / 32;
  __shared__ float s_m[W], s_S[W], s_U[W];
  __shared__ float4 s_part;
  __shared__ Targets s_y;
  __shared__ TopShared s_top;
  __shared__ uint32_t s_best[kParts<NT> * NT];
  const unsigned rank = cluster_ctarank();
  unsigned nc;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nc));
  const int64_t t = blockIdx.x / nc;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  const T* x = static_cast<const T*>(a.x) + t * a.ld;
  const Row<T> row(x, a.V);
  // this block's whole words, and the partial ones that are its
  const int per = (row.nw + static_cast<int>(nc) - 1) / static_cast<int>(nc);
  const int w0 = min(row.nw, static_cast<int>(rank) * per), w1 = min(row.nw, w0 + per);
  const int first = max(w0, row.head ? 1 : 0), end = min(w1, row.nw - (row.tail ? 1 : 0));
  const int edge0 = row.head && w0 == 0 ? 0 : -1;
  const int edge1 = row.tail && w0 < row.nw && w1 == row.nw ? row.nw - 1 : -1;
  for (int j = threadIdx.x; j < a.m; j += NT) {
    const int y = target(a, t, j, rank == 0);
    s_y.y[j] = y;
    s_y.x[j] = y >= 0 ? value(x + y) : 0.f;
    s_y.g[j] = GRAD && y >= 0 && a.dlogp != nullptr ? a.dlogp[t * a.m + j] : 0.f;
  }

  Sums<ENT> sums;
  // words from i0 up to `to`, NT apart
  auto add_words = [&](int i0, int to) {
    for (; i0 + (U - 1) * NT < to; i0 += NT * U) {
      uint4 q[U];
#pragma unroll
      for (int u = 0; u < U; ++u) q[u] = row.word(i0 + u * NT);
#pragma unroll
      for (int u = 0; u < U; ++u) sums.template add<T>(q[u], a.c, a.floor);
    }
    if (i0 < to) {
      uint4 q[U - 1];
#pragma unroll
      for (int u = 0; u < U - 1; ++u)
        if (i0 + u * NT < to) q[u] = row.word(i0 + u * NT);
#pragma unroll
      for (int u = 0; u < U - 1; ++u)
        if (i0 + u * NT < to) sums.template add<T>(q[u], a.c, a.floor);
    }
  };
  // words of a part: whole groups of loads, so that the parts cost the loop nothing
  const int step = (max(end - first, 0) + kParts<NT> * NT * U - 1) / (kParts<NT> * NT * U) * (NT * U);
  if (TOP) {
    float all = -INFINITY;
#pragma unroll 1
    for (int i = 0; i < kParts<NT>; ++i) {
      sums.mx = -INFINITY;
      add_words(first + i * step + static_cast<int>(threadIdx.x), min(end, first + (i + 1) * step));
      s_best[i * NT + threadIdx.x] = sums.mx > -INFINITY ? ordered(sums.mx) : 0u;
      all = fmaxf(all, sums.mx);
    }
    sums.mx = all;
  } else {
    add_words(first + static_cast<int>(threadIdx.x), end);
  }
  if (threadIdx.x < 2) {
    const int i = threadIdx.x == 0 ? edge0 : edge1;
    if (i >= 0) sums.template add<T>(row.partial(i), a.c, a.floor);
  }

  // sums of the threads' S and U over the block, in every thread
  auto block_sums = [&](float& S, float& Us) {
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, i);
      if (ENT) Us += __shfl_xor_sync(0xffffffffu, Us, i);
    }
    if (W == 1) return;
    if (lane == 0) s_S[warp] = S, s_U[warp] = Us;
    __syncthreads();
    S = Us = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) S += s_S[i], Us += ENT ? s_U[i] : 0.f;
  };
  float M = sums.mx;
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, i));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < W; ++i) M = fmaxf(M, s_m[i]);
  float S = sum2(sums.S), Us = ENT ? sum2(sums.U) : 0.f;
  const float block_at = fmaxf(M * a.c, kUnset);
  relate(sums.at, block_at, S, Us);
  block_sums(S, Us);
  if (TOP) block_top<T, NT>(s_top, s_best, row, first, end, step, edge0, edge1, ordered(M), a.top);

  // over the cluster
  if (nc > 1) {
    if (threadIdx.x == 0) s_part = make_float4(M, S, Us, block_at);
    cluster_sync();
    float pm[kMaxCluster], ps[kMaxCluster], pu[kMaxCluster], pa[kMaxCluster];
#pragma unroll
    for (unsigned r = 0; r < kMaxCluster; ++r) {
      pm[r] = -INFINITY, ps[r] = pu[r] = 0.f, pa[r] = kUnset;
      if (r < nc) {
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(pm[r]), "=f"(ps[r]), "=f"(pu[r]), "=f"(pa[r])
                     : "r"(mapa_shared(smem_u32(&s_part), r))
                     : "memory");
      }
      M = fmaxf(M, pm[r]);
    }
    S = Us = 0.f;
    const float at = fmaxf(M * a.c, kUnset);
#pragma unroll
    for (unsigned r = 0; r < kMaxCluster; ++r) {
      relate(pa[r], at, ps[r], pu[r]);
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
      for (int i = threadIdx.x; i < a.top; i += NT) s_top.out[i] = 0;
      __syncthreads();
      // empty places (0) of several blocks are equal: they are left out
      for (int i = threadIdx.x; i < total; i += NT) {
        const uint64_t key = s_top.cand[i];
        int place = 0;
        for (int j = 0; j < total; ++j) place += s_top.cand[j] > key;
        if (key != 0 && place < a.top) s_top.out[place] = key;
      }
      __syncthreads();
    }
  }
  const Shift shift(M > -INFINITY ? M : 0.f, a.c);
  if (shift.extreme) {  // the same for the whole cluster
    S = Us = 0.f;
    for (int i = first + static_cast<int>(threadIdx.x); i < end; i += NT) add_extreme<T>(row.word(i), shift, S, Us);
    if (threadIdx.x < 2) {
      const int i = threadIdx.x == 0 ? edge0 : edge1;
      if (i >= 0) add_extreme<T>(row.partial(i), shift, S, Us);
    }
    __syncthreads();  // s_S was read above
    block_sums(S, Us);
    if (nc > 1) {
      cluster_sync();  // s_part was read by every block
      if (threadIdx.x == 0) s_part = make_float4(M, S, Us, 0.f);
      cluster_sync();
      S = Us = 0.f;
      for (unsigned r = 0; r < nc; ++r) {
        float4 p;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(p.x), "=f"(p.y), "=f"(p.z), "=f"(p.w)
                     : "r"(mapa_shared(smem_u32(&s_part), r))
                     : "memory");
        S += p.y;
        Us += p.z;
      }
    }
  }

  if (nc > 1) cluster_arrive();  // has read the others' shared memory
  const bool empty = S == 0.f;
  const float log_S = logf(S);
  if (rank == 0) {
    for (int j = threadIdx.x; j < a.m; j += NT)
      a.logp[t * a.m + j] = s_y.y[j] < 0 ? 0.f
                            : empty      ? -INFINITY
                                         : shift.log_share(s_y.x[j], log_S, a.inv_temp);
    if (threadIdx.x == 0) {
      a.stats[2 * t] = shift.M;
      a.stats[2 * t + 1] = S;
      if (a.lse != nullptr) a.lse[t] = empty ? -INFINITY : fmaf(shift.M, a.inv_temp, log_S);
      if (ENT && a.entropy != nullptr) a.entropy[t] = empty ? 0.f : log_S - kLn2 * Us / S;
    }
    if (TOP && static_cast<int>(threadIdx.x) < a.top) {
      const uint64_t key = s_top.out[threadIdx.x];
      const int64_t at = t * a.top + threadIdx.x;
      if (a.top_ids != nullptr) a.top_ids[at] = key != 0 ? static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
      if (a.top_logp != nullptr)
        a.top_logp[at] = key == 0 ? -INFINITY
                                  : shift.log_share(from_ordered(static_cast<uint32_t>(key >> 32)), log_S, a.inv_temp);
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
    // where a row takes a cluster, the rows in flight fill the L2: what is read for the second
    // time may leave it first (4096 x 151936: 438 us, 446 otherwise; 16384 x 32000, a block
    // each: 334, 322)
    gradient_words<T, NT, U, ENT>(row, drow, threadIdx.x, first, end, edge0, edge1, a.same != 0, zero, shift,
                                  a.floor, k.A, k.B, [&](int i) {
                                    return nc > 1 ? __ldcs(row.at(i)) : *row.at(i);
                                  });
    __syncthreads();
    if (!zero)
      for (int j = threadIdx.x; j < a.m; j += NT) {
        const int y = s_y.y[j], w = (y + row.h) / Row<T>::E;
        if (y >= 0 && w >= w0 && w < w1) put_target(s_y, j, a.m, drow, shift, k.A, k.B, a.inv_temp);
      }
  }
  if (nc > 1) cluster_wait();  // no block leaves while its shared memory is read
}

// The gradient alone: a warp takes a unit of kBwdWords * `turns` words a lane, so that rows
// of any length fill the SMs and no thread waits for another warp (4096 x 151936: 357 us).
constexpr int kBwdThreads = 256, kBwdWarps = kBwdThreads / 32, kBwdWords = 4;
template <typename T, bool ENT>
__global__ void __launch_bounds__(kBwdThreads, 5) logprob_bwd_kernel(const Args a, int turns, int chunks,
                                                                    int64_t units) {
  __shared__ Targets s_targets[kBwdWarps];
  const int lane = threadIdx.x & 31;
  Targets& s_y = s_targets[threadIdx.x >> 5];
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kBwdWarps;
  pdl_wait();
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * kBwdWarps + (threadIdx.x >> 5); unit < units;
       unit += warps) {
    const int64_t t = (unit >> 32) == 0 ? static_cast<int64_t>(static_cast<uint32_t>(unit) / static_cast<uint32_t>(chunks))
                                        : unit / chunks;
    const int chunk = static_cast<int>(unit - t * chunks);
    const T* x = static_cast<const T*>(a.x) + t * a.ld;
    const Row<T> row(x, a.V);
    const int w0 = chunk * 32 * kBwdWords * turns, w1 = min(row.nw, w0 + 32 * kBwdWords * turns);
    if (w0 >= w1) continue;
    const int first = max(w0, row.head ? 1 : 0), end = min(w1, row.nw - (row.tail ? 1 : 0));
    const int edge0 = row.head && w0 == 0 ? 0 : -1, edge1 = row.tail && w1 == row.nw ? row.nw - 1 : -1;
    const float M = a.stats_in[2 * t], S = a.stats_in[2 * t + 1];
    const float dent = ENT ? a.dent[t] : 0.f, dlse = a.dlse != nullptr ? a.dlse[t] : 0.f;
    const float less = ENT ? logf(S) - a.entropy_in[t] : 0.f;
    auto mine = [&](int y) {
      const int w = (y + row.h) / Row<T>::E;
      return y >= 0 && w >= w0 && w < w1;
    };
    float sum_g = 0.f;
    bool some = false, here = false;  // a gradient that is not zero; a target in this unit
    for (int j = lane; j < (a.m + 31 & ~31); j += 32) {
      const int y = j < a.m ? target(a, t, j, false) : -1;
      float g = y >= 0 && a.dlogp != nullptr ? a.dlogp[t * a.m + j] : 0.f;
      some |= __any_sync(0xffffffffu, g != 0.f);
      here |= __any_sync(0xffffffffu, mine(y));
      if (a.m > 1) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) g += __shfl_xor_sync(0xffffffffu, g, o);
      }
      sum_g += __shfl_sync(0xffffffffu, g, 0);
    }
    const bool zero = S == 0.f || !(some || dent != 0.f || dlse != 0.f);
    const Coefs k = coefs(sum_g, dent, dlse, S, less, a.inv_temp);
    const Shift shift(M, a.c);
    here &= !zero;
    if (here) {
      // logits of targets are read before their words are overwritten (dlogits may be logits)
      __syncwarp();
      for (int j = lane; j < a.m; j += 32) {
        const int y = target(a, t, j, false);
        s_y.y[j] = mine(y) ? y : -1;
        s_y.g[j] = y >= 0 && a.dlogp != nullptr ? a.dlogp[t * a.m + j] : 0.f;
        s_y.x[j] = mine(y) ? value(x + y) : 0.f;
      }
      __syncwarp();
    }
    T* drow = static_cast<T*>(a.dx) + t * a.dld;
    gradient_words<T, 32, kBwdWords, ENT>(row, drow, lane, first, end, edge0, edge1, a.same != 0, zero, shift,
                                          a.floor, k.A, k.B, [&](int i) { return row.word(i); });
    if (here) {
      __syncwarp();
      for (int j = lane; j < a.m; j += 32)
        if (s_y.y[j] >= 0) put_target(s_y, j, a.m, drow, shift, k.A, k.B, a.inv_temp);
    }
  }
}

// ---- launches -----------------------------------------------------------------------------
// Threads of a block: about 8 words each, 256 where a row is longer (128 in one case below),
// 512 where there are few rows (one of 151936 logits, its 20 likeliest: 8.2 us, with 256 threads 9.9).  Blocks of a row:
// one where that gives four for each SM, more, up to eight, where there are fewer rows.
// With the gradient also as many as it takes for the rows in flight, five blocks to an
// SM, to stay in the L2 until their second reading.
constexpr int kLane = 256, kSmall = 2048;       // words of a block up to which it has 32, 128 threads
constexpr int64_t kInFlight = int64_t(80) << 20;

template <typename T, int NT, int MINB, bool GRAD, int U = 4>
cudaError_t rows(const Args& a, unsigned cluster, cudaStream_t s) {
  const bool ent = a.entropy != nullptr || a.dent != nullptr;
  auto kernel = a.top > 0 ? (ent ? logprob_kernel<T, NT, MINB, U, true, true, GRAD>
                                 : logprob_kernel<T, NT, MINB, U, true, false, GRAD>)
                          : (ent ? logprob_kernel<T, NT, MINB, U, false, true, GRAD>
                                 : logprob_kernel<T, NT, MINB, U, false, false, GRAD>);
  return launch_pdl_cluster(kernel, dim3(static_cast<unsigned>(a.T) * cluster), dim3(NT), 0, s, cluster, a);
}
template <typename T>
int64_t row_words(const Args& a) {  // a row's most
  return (static_cast<int64_t>(a.V) + 2 * Row<T>::E - 2) / Row<T>::E;
}
template <typename T, bool GRAD>
cudaError_t launch_rows(const Args& a, cudaStream_t s) {
  const int64_t words = row_words<T>(a);
  unsigned cluster = 1;
  while (cluster < kMaxCluster &&
         ((static_cast<int64_t>(a.T) * cluster < 4 * kSMs && words > kSmall / 2 * static_cast<int64_t>(cluster)) ||
          (GRAD && words > kSmall && words * 16 * (5 * kSMs / cluster) > kInFlight)))
    cluster *= 2;
  const int64_t each = (words + cluster - 1) / cluster;
  // so few rows that every block has half an SM: all of a thread's loads at once.  (256, as not
  // every SM has a place in a cluster of eight: 38 rows in 304 blocks take two turns, 14.6 us
  // against 11.4 with 256 threads.)
  if (each > kSmall / 2 && static_cast<int64_t>(a.T) * cluster <= 256)
    return rows<T, 512, 2, GRAD, 8>(a, cluster, s);
  // Rows that blocks of 128 threads have places for at once, and those of 256 do not: one
  // turn instead of two (900 rows of 151936: 50 us, 59; 620, which 256 threads have places
  // for: 44, 37).  With a list, whose second reading is by half as many threads, while rows,
  // words and tokens listed are few.  Of 175 points (1 to 32 tokens, 620 to 1200 rows of
  // 20000 to 151936) the rule takes the faster form or one within 2 % but for five (3 to 9 %):
  // 900x32000, 5 tokens 21 us, 27; 1024x100352, 5 tokens 47.6, 48.0; 1200x128000, 5 tokens
  // 66, 60; 900x50257, 20 tokens 32, 34, 32 tokens 37, 35.
  const bool one_turn = !GRAD && cluster == 1 && a.T <= 8 * kSMs && a.T > (a.top > 0 ? 4 : 5) * kSMs &&
                        (a.top == 0 || a.T * words * (a.top + 6) <= 145 << 20);
  return each <= kLane                 ? rows<T, 32, 20, GRAD>(a, cluster, s)
         : each <= kSmall || one_turn ? rows<T, 128, 8, GRAD>(a, cluster, s)
         : a.top > 0                  ? rows<T, 256, 4, GRAD>(a, cluster, s)
                                      : rows<T, 256, 5, GRAD>(a, cluster, s);
}
template <typename T>
cudaError_t launch_bwd(const Args& a, cudaStream_t s) {
  const int64_t words = row_words<T>(a);
  const int turns = words >= 4096 ? 4 : 1;
  const int64_t unit = 32 * kBwdWords * turns, chunks = (words + unit - 1) / unit, units = chunks * a.T;
  const int64_t blocks = (units + kBwdWarps - 1) / kBwdWarps;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(blocks, 0x7FFFFFFF));
  return launch_pdl(a.dent != nullptr ? logprob_bwd_kernel<T, true> : logprob_bwd_kernel<T, false>, dim3(grid),
                    dim3(kBwdThreads), 0, s, a, turns, static_cast<int>(chunks), units);
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
  if (!(q->inv_temp >= 1e-30f && q->inv_temp <= 1e30f)) return bad("inv_temp must be in 1e-30 .. 1e30");
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
  const float low = kFloor / a.c;  // inv_temp >= 1e-30: above the types' lowest value
  std::memcpy(&a.floor, &low, 4);
  if (q->type == MOE_BF16) a.floor = (a.floor >> 16) | (a.floor & 0xFFFF0000u);
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
  const cudaError_t e = desc->type == MOE_BF16 ? launch_rows<bf16_t, false>(a, stream)
                                               : launch_rows<float, false>(a, stream);
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
  const cudaError_t e = desc->type == MOE_BF16 ? launch_rows<bf16_t, true>(a, stream)
                                               : launch_rows<float, true>(a, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
