// One AdamW step over many tensors at once, moments in 32 bits or in 8, with
// the clip by the global gradient norm.
//   g = c grad,  c = grad_scale min(1, max_norm / (norm + 1e-6)),  norm = |grad_scale grad|_2
//   m = b1 m + (1 - b1) g,  v = b2 v + ((1 - b2) g) g,  root = sqrt(v)
//   p = p (1 - lr wd) - lr/(1 - b1^t) (m / (root / sqrt(1 - b2^t) + eps))
// in fp32, each operation rounded by itself (no contraction), so that the
// results do not depend on how a launch is cut.
//
// 8-bit moments: m and root are held as e4m3 values (1-4-3 bits, largest 448,
// subnormals down to 2^-9) times a power-of-two scale shared by a block of 256
// consecutive values, its exponent held as E8M0 byte: the block's largest
// value lands in [128, 256).  root rather than v, since v's exponents span
// twice as many bits.  Values are rounded down to the grid after adding
// u 2^-20 of a grid step, u the top 20 bits of i I + t T mod 2^32 (i the
// value's index in its tensor, t the step, T and I odd, the fractional parts
// of the golden ratio and of the square root of 2): over the steps the
// thresholds of a value are spread evenly, so an update far below a grid step
// (v moves by 0.1 % a step, the grid is 6-12 % apart) passes in its due share
// of the steps, where rounding to nearest would lose it every time.  A root
// above zero is kept above zero (it divides).
//
// The sum of squares is kept as a pair of floats (the rounding errors of each
// product and each sum in the second), about 46 significant bits: the norm,
// rounded to fp32, does not depend on the order either, to all purposes.
//
// One pass; a block of threads takes chunks of 2048 values, 8 for each thread.
// 32-bit moments are bound by memory: 52 M bf16 parameters with fp32 gradients and
// master copies take 274 us with the clip (0.96 of the rate of a plain copy on what
// both passes read and write, some of it in the L2; 300 us with 16-byte accesses,
// which touch every line of fp32 values by halves).  With 8-bit moments the same take
// 164 us, 5.8 TB/s; 16 M bf16 values with bf16 gradients and no master copies 41 us,
// 4 TB/s (what holds them there is not shown: of 40 such tensors, 4 M values, an SM
// issues in 40 % of its cycles).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cuda_fp8.h>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kBlock = MOE_ADAMW_BLOCK;        // values per scale: 8 for each lane of a warp
constexpr int kThreads = 256;
constexpr int kChunk = kThreads * 8;           // values of one pass of a block of threads
constexpr int kNormBlocks = 8 * kSMs;          // rows of partial sums per norm launch
constexpr uint32_t kDitherT = 2654435769u, kDitherI = 1779033703u;

struct Tensor {
  void* p;
  float* master;
  const void* g;
  void* m;
  void* v;
  uint8_t* sc;
  int64_t n;
  float keep, lr;  // 1 - lr wd; lr / (1 - b1^t)
  int vec;         // 1: all pointers allow 16-byte accesses, 2: fp32 ones 32-byte accesses
};
struct Consts {
  float b1, c1, b2, c2, correct, eps, grad_scale, max_norm;
  float zero;            // -0
  uint32_t dither;       // t T
  const float2* part;    // partial sums of squares (value, rest), NULL: not needed
  int nparts, skip;
  float* norm_out;
};
// Tables travel as kernel arguments (constant memory, no copy, no lifetime):
// three sizes up to the 32 KB limit, as a launch copies all of it (40 tensors:
// 13.6 us of host time with the largest, 12.0 with the middle one).
constexpr int kFew = 24, kSome = 96, kMany = 400;
// The tensors' first chunks, and for every 2^shift chunks the tensor of the first
// of them, which leaves little of the table to search.
template <int MAX>
struct Starts {
  static constexpr int kHints = MAX <= 64 ? 64 : MAX <= 256 ? 256 : 1024;
  int n, chunks, shift;
  int start[MAX];
  uint16_t hint[kHints + 1];

  void clear() { n = chunks = 0; }
  bool full(int64_t ch) const { return n == MAX || chunks + ch > (int64_t(1) << 30); }
  int add(int64_t ch) {  // a tensor of ch chunks; its number
    start[n] = chunks;
    chunks += static_cast<int>(ch);
    return n++;
  }
  void close() {
    shift = 0;
    while (((chunks - 1) >> shift) >= kHints) ++shift;
    const int used = ((chunks - 1) >> shift) + 1;
    for (int b = 0, t = 0; b < used; ++b) {
      while (t + 1 < n && start[t + 1] <= b << shift) ++t;
      hint[b] = static_cast<uint16_t>(t);
    }
    hint[used] = static_cast<uint16_t>(n - 1);
  }
  // The tensor that chunk ch belongs to: the last that starts at or before it.
  __device__ __forceinline__ int of(int ch) const {
    const int b = ch >> shift;
    int lo = hint[b], hi = hint[b + 1] + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= ch) lo = mid;
      else hi = mid;
    }
    return lo;
  }
};
template <int MAX>
struct Table {
  Consts c;
  Starts<MAX> s;
  Tensor t[MAX];
};
struct NormTensor {
  const void* g;
  int64_t n2;      // 2 n, + 1 for bf16
};
constexpr int kNormFew = 64, kNormSome = 256, kNormMany = 1200;
template <int MAX>
struct NormTable {
  float zero;  // -0
  float2* part;
  Starts<MAX> s;
  NormTensor t[MAX];
};

// Packed product that no later sum is contracted with: the assembler makes one
// fma of a packed mul and add in spite of their rounding modifiers, so the
// product is an fma itself, with a zero that it cannot know (-0, so that every
// product comes through as it is).
struct Product {
  f2 zero;
  __device__ __forceinline__ f2 operator()(f2 a, f2 b) const { return fma2(a, b, zero); }
};

// Eight values from index i on (those past n read as 0 / are not written).
// vec: all eight are there and 16-byte accesses will do; WIDE: 32-byte ones.
template <bool WIDE, typename T>
__device__ __forceinline__ void take(const T* p, int64_t i, int64_t n, bool vec, f2 (&f)[4]) {
  Raw8<T> r;
  if (vec) {
    if constexpr (WIDE && sizeof(T) == 4) load8_wide(p + i, r);
    else load8<true>(p + i, 0, 8, r);
    widen(r, f);
    return;
  }
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = 0.f;
    if (i + e < n) {
      if constexpr (sizeof(T) == 2)
        x[e] = __uint_as_float(static_cast<uint32_t>(p[i + e].bits) << 16);
      else
        x[e] = p[i + e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) f[e] = pk(x[2 * e], x[2 * e + 1]);
}
template <bool WIDE, typename T>
__device__ __forceinline__ void give(T* p, int64_t i, int64_t n, bool vec, const f2 (&f)[4]) {
  Raw8<T> r;
  narrow(f, r);
  if (vec) {
    if constexpr (WIDE && sizeof(T) == 4) store8_wide(p + i, r);
    else store8<true>(p + i, 0, 8, r);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) {
      if constexpr (sizeof(T) == 2) {
        const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
        p[i + e].bits = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
      } else {
        const float2 x = unpk(f[e >> 1]);
        p[i + e] = e & 1 ? x.y : x.x;
      }
    }
}
// Eight code bytes.
__device__ __forceinline__ uint2 get_codes(const uint8_t* p, int64_t i, int64_t n, bool vec) {
  if (vec) return *reinterpret_cast<const uint2*>(p + i);
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) w[e >> 2] |= static_cast<uint32_t>(p[i + e]) << (8 * (e & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void set_codes(uint8_t* p, int64_t i, int64_t n, bool vec, uint2 q) {
  if (vec) {
    *reinterpret_cast<uint2*>(p + i) = q;
    return;
  }
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (i + e < n) p[i + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
}
__device__ __forceinline__ void decode8(uint2 q, float scale, f2 (&f)[4]) {
  const uint32_t w[2] = {q.x, q.y};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>(w[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
    const float2 x = __half22float2(__half2(hr));
    f[h] = mul2(pk(x.x, x.y), pk(scale));  // exact
  }
}
// E8M0 byte of a block whose largest magnitude has the bits `top`.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const int b = static_cast<int>(top >> 23) - 7;
  return b < 8 ? 8u : b > 248 ? 248u : static_cast<uint32_t>(b);
}
// Top bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}
// Largest (a NaN is the largest) and least (a NaN counts only among NaNs)
// magnitude of eight values, three at a time.
__device__ __forceinline__ float most3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float least3(float a, float b, float c) {
  float r;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t most8(const float (&x)[8]) {
  return __float_as_uint(most3(most3(x[0], x[1], x[2]), most3(x[3], x[4], x[5]), most3(x[6], x[7], x[7])));
}
__device__ __forceinline__ float least8(const float (&x)[8]) {
  return least3(least3(x[0], x[1], x[2]), least3(x[3], x[4], x[5]), least3(x[6], x[7], x[7]));
}
// The eight codes of this lane: m with its sign, root not below 1 where positive.
// least_v: the least of the roots' squares.
__device__ __forceinline__ void encode8(const float (&m)[8], const float (&root)[8], float least_v,
                                        uint32_t u, uint32_t bm, uint32_t bv, uint2& qm, uint2& qr) {
  // A normal value's code is in place after one addition: bits 20-26 of the
  // rebased, dithered word.  Below the smallest normal value (2^-6 scale), adding
  // that value first makes the grid linear; its exponent comes off again.  A warp
  // looks after such values where it has one: m or root below 2^-14 of their
  // block's largest.
  const uint32_t sub_m = (bm - 7u) << 23, sub_r = (bv - 7u) << 23;
  const float low_m = __uint_as_float((bm - 6u) << 23), low_r = __uint_as_float((bv - 6u) << 23);
  const float low_v = fmaxf(1.0001f * low_r * low_r, 0x1p-126f);  // the square may vanish
  uint32_t wm[8], wr[8];
  if (__all_sync(0xffffffffu, least8(m) >= low_m)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t x = __float_as_uint(m[e]) + ((u + e * kDitherI) >> 12) - sub_m;
      wm[e] = ((x << 4) & 0x7FFFFFFFu) | (x & 0x80000000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool below = fabsf(m[e]) < low_m;
      const uint32_t x = __float_as_uint(below ? __fadd_rn(m[e], m[e] < 0.f ? -low_m : low_m) : m[e]) +
                         ((u + e * kDitherI) >> 12) - (below ? sub_m + (1u << 23) : sub_m);
      wm[e] = ((x << 4) & 0x7FFFFFFFu) | (x & 0x80000000u);
    }
  }
  if (__all_sync(0xffffffffu, least_v >= low_v)) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      wr[e] = (__float_as_uint(root[e]) + (0xFFFFFu - ((u + e * kDitherI) >> 12)) - sub_r) << 4;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool below = root[e] < low_r;
      wr[e] = (__float_as_uint(below ? __fadd_rn(root[e], low_r) : root[e]) +
               (0xFFFFFu - ((u + e * kDitherI) >> 12)) - (below ? sub_r + (1u << 23) : sub_r)) << 4;
      if (root[e] > 0.f) wr[e] = max(wr[e], 1u << 24);
    }
  }
  qm = make_uint2(top_bytes(wm[0], wm[1], wm[2], wm[3]), top_bytes(wm[4], wm[5], wm[6], wm[7]));
  qr = make_uint2(top_bytes(wr[0], wr[1], wr[2], wr[3]), top_bytes(wr[4], wr[5], wr[6], wr[7]));
}

// Sums held as a pair of floats (value, rest), since 64-bit adds are some 60
// times slower here: the exact error of each fp32 addition goes to the rest.  A value
// that is not finite has no rest (its error would be Inf - Inf), so that an infinite
// sum stays infinite.
__device__ __forceinline__ float2 add_pair(float2 a, float2 b) {
  const float s = __fadd_rn(a.x, b.x), t = __fsub_rn(s, a.x);
  if (!(fabsf(s) < INFINITY)) return make_float2(s, 0.f);
  const float err = __fadd_rn(__fsub_rn(a.x, __fsub_rn(s, t)), __fsub_rn(b.x, t));
  const float rest = __fadd_rn(err, __fadd_rn(a.y, b.y));
  const float v = __fadd_rn(s, rest);
  return make_float2(v, __fsub_rn(rest, __fsub_rn(v, s)));
}
__device__ __forceinline__ float2 warp_pair(float2 a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = add_pair(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.y, o)));
  return a;
}
// The sum over the block, in every thread.
__device__ __forceinline__ float2 block_pair(float2 a, float2* s_warp) {
  a = warp_pair(a);
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = a;
  __syncthreads();
  a = s_warp[0];
#pragma unroll
  for (int i = 1; i < kThreads / 32; ++i) a = add_pair(a, s_warp[i]);
  return a;
}
__device__ __forceinline__ float root_of_pair(float2 a) {
  const float s = __fsqrt_rn(a.x);
  if (!(s > 0.f && s < INFINITY)) return s;
  const float r = __fadd_rn(__fmaf_rn(-s, s, a.x), a.y);
  return __fmaf_rn(r, __fdiv_rn(0.5f, s), s);
}

// Square root and quotient, rounded to nearest: an approximate reciprocal
// (square root), one Newton step, and a last correction by the exact residual
// (Markstein, IBM J. Res. Dev. 34, 1990).  x >= 0; d from 2^-100 to 2^120.
template <bool NORMAL>
__device__ __forceinline__ float approx_rsqrt(float x) {
  float r;
  if (NORMAL) asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  else asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float approx_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 root2(f2 x, f2 y, const Product& mul) {  // y: about 1 / sqrt(x)
  const f2 s = mul(x, y), nh = mul(y, pk(-0.5f));
  const f2 e = fma2(s, nh, pk(0.5f));
  const f2 nh1 = fma2(nh, e, nh), s1 = fma2(s, e, s);
  return fma2(fma2(s1, s1, mul(x, pk(-1.f))), nh1, s1);
}
// The roots of eight values, whose least is `least`: where it is a normal number
// nothing below one need be looked after, nor zeros.
__device__ __forceinline__ void roots8(const f2 (&x)[4], float least, const Product& mul, f2 (&root)[4]) {
  if (least >= 0x1p-126f) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = unpk(x[e]);
      root[e] = root2(x[e], pk(approx_rsqrt<true>(v.x), approx_rsqrt<true>(v.y)), mul);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 v = unpk(x[e]);  // 0: a finite factor, so that 0 comes out
      root[e] = root2(x[e], pk(approx_rsqrt<false>(fmaxf(v.x, 1e-45f)), approx_rsqrt<false>(fmaxf(v.y, 1e-45f))), mul);
    }
  }
}
__device__ __forceinline__ f2 ratio2(f2 n, f2 d, const Product& mul) {
  // 2^120 where v overflowed: root2 makes NaN of an infinite v, and fminf drops it
  const float2 v = unpk(d);
  const float x = fminf(v.x, 0x1p120f), y = fminf(v.y, 0x1p120f);
  const f2 r = pk(approx_rcp(x), approx_rcp(y)), nd = pk(-x, -y);
  const f2 r1 = fma2(r, fma2(nd, r, pk(1.f)), r);
  const f2 q = mul(n, r1);
  return fma2(fma2(nd, q, n), r1, q);
}

// Eight values of each thread, from index i of the tensor t on.
template <typename PT, typename GT, bool MASTER, bool EIGHT, bool WIDE>
__device__ __forceinline__ void update8(const Consts& c, const Tensor& t, int64_t i, bool vec, float coef,
                                        const Product& mul) {
  const int64_t n = t.n;
  f2 p[4], g[4], m[4], v[4], root[4];
  take<WIDE>(static_cast<const GT*>(t.g), i, n, vec, g);
  if (MASTER) take<WIDE>(t.master, i, n, vec, p);
  else take<WIDE>(static_cast<const PT*>(t.p), i, n, vec, p);
  const int64_t blk = i / kBlock;  // the same for the whole warp
  if constexpr (EIGHT) {
    uint32_t bm = 0, bv = 0;
    if (blk * kBlock < n) {
      bm = t.sc[2 * blk];
      bv = t.sc[2 * blk + 1];
    }
    const uint2 qm = get_codes(static_cast<const uint8_t*>(t.m), i, n, vec);
    const uint2 qv = get_codes(static_cast<const uint8_t*>(t.v), i, n, vec);
    decode8(qm, __uint_as_float(bm << 23), m);
    decode8(qv, __uint_as_float(bv << 23), v);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = mul(v[e], v[e]);
  } else {
    take<WIDE>(static_cast<const float*>(t.m), i, n, vec, m);
    take<WIDE>(static_cast<const float*>(t.v), i, n, vec, v);
  }
  const f2 coef2 = pk(coef), b1 = pk(c.b1), c1 = pk(c.c1), b2 = pk(c.b2), c2 = pk(c.c2),
           keep = pk(t.keep), nlr = pk(-t.lr);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    g[e] = mul(g[e], coef2);
    m[e] = add2(mul(b1, m[e]), mul(c1, g[e]));
    v[e] = add2(mul(b2, v[e]), mul(mul(c2, g[e]), g[e]));
  }
  float vv[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = unpk(v[e]);
    vv[2 * e] = x.x; vv[2 * e + 1] = x.y;
  }
  const float least_v = least8(vv);
  roots8(v, least_v, mul, root);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const f2 upd = ratio2(m[e], add2(mul(root[e], pk(c.correct)), pk(c.eps)), mul);
    p[e] = add2(mul(p[e], keep), mul(nlr, upd));
  }
  if constexpr (EIGHT) {
    float mm[8], rr[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = unpk(m[e]), y = unpk(root[e]);
      mm[2 * e] = x.x; mm[2 * e + 1] = x.y;
      rr[2 * e] = y.x; rr[2 * e + 1] = y.y;
    }
    // values past n are 0: they do not raise the maximum
    const uint32_t bm = scale_byte(__reduce_max_sync(0xffffffffu, most8(mm)));
    const uint32_t bv = scale_byte(__reduce_max_sync(0xffffffffu, most8(rr)));
    uint2 qm, qr;
    encode8(mm, rr, least_v, static_cast<uint32_t>(i) * kDitherI + c.dither, bm, bv, qm, qr);
    set_codes(static_cast<uint8_t*>(t.m), i, n, vec, qm);
    set_codes(static_cast<uint8_t*>(t.v), i, n, vec, qr);
    if ((threadIdx.x & 31) == 0 && i < n) {
      t.sc[2 * blk] = static_cast<uint8_t>(bm);
      t.sc[2 * blk + 1] = static_cast<uint8_t>(bv);
    }
  } else {
    give<WIDE>(static_cast<float*>(t.m), i, n, vec, m);
    give<WIDE>(static_cast<float*>(t.v), i, n, vec, v);
  }
  give<WIDE>(static_cast<PT*>(t.p), i, n, vec, p);
  if (MASTER) give<WIDE>(t.master, i, n, vec, p);
}

template <typename PT, typename GT, bool MASTER, bool EIGHT, int MAX>
__global__ void __launch_bounds__(kThreads, EIGHT ? 5 : 4) adamw_kernel(const __grid_constant__ Table<MAX> tab) {
  const Consts& c = tab.c;
  const Product mul{pk(c.zero)};
  float coef = c.grad_scale;
  pdl_wait();
  if (c.part != nullptr) {  // the norm: every block adds the same partials in the same order
    __shared__ float2 s_sum[kThreads / 32];
    float2 s = make_float2(0.f, 0.f);
    for (int i = threadIdx.x; i < c.nparts; i += kThreads) s = add_pair(s, c.part[i]);
    const float norm = __fmul_rn(root_of_pair(block_pair(s, s_sum)), fabsf(c.grad_scale));
    if (c.norm_out != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *c.norm_out = norm;
    if (c.skip && !(norm <= 3.402823466e38f)) return;  // Inf or NaN: nothing changes
    if (c.max_norm > 0.f) {
      const float q = __fdiv_rn(c.max_norm, __fadd_rn(norm, 1e-6f));
      coef = __fmul_rn(coef, q >= 1.f ? 1.f : q);  // a NaN norm stays NaN
    }
  }
  // Backwards: after a norm the gradients' end is what is left of them in the L2.
  for (int ch = tab.s.chunks - 1 - static_cast<int>(blockIdx.x); ch >= 0; ch -= gridDim.x) {
    const int ti = tab.s.of(ch);
    const Tensor& t = tab.t[ti];
    const int64_t first = static_cast<int64_t>(ch - tab.s.start[ti]) * kChunk, i = first + threadIdx.x * 8;
    if (t.vec == 2 && first + kChunk <= t.n)  // the same for all threads: they vote
      update8<PT, GT, MASTER, EIGHT, true>(c, t, i, true, coef, mul);
    else
      update8<PT, GT, MASTER, EIGHT, false>(c, t, i, t.vec != 0 && i + 8 <= t.n, coef, mul);
  }
}

// hi + lo += x^2, elementwise: the exact error of the product and of the sum
// with hi go to lo.
__device__ __forceinline__ void add_square(f2 x, f2& hi, f2& lo, const Product& mul) {
  const f2 minus = pk(-1.f);
  const f2 p = mul(x, x);
  const f2 e = fma2(x, x, mul(p, minus));
  const f2 s = add2(hi, p);
  const f2 b = fma2(hi, minus, s);                                    // s - hi
  const f2 err = add2(fma2(fma2(b, minus, s), minus, hi), fma2(b, minus, p));
  hi = s;
  lo = add2(lo, add2(err, e));
}

template <int MAX>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ NormTable<MAX> tab) {
  __shared__ float2 s_sum[kThreads / 32];
  pdl_wait();
  const Product mul{pk(tab.zero)};
  f2 hi = pk(0.f), lo = pk(0.f);
  for (int ch = blockIdx.x; ch < tab.s.chunks; ch += gridDim.x) {
    const int ti = tab.s.of(ch);
    const NormTensor& t = tab.t[ti];
    const int64_t i = static_cast<int64_t>(ch - tab.s.start[ti]) * kChunk + threadIdx.x * 8, n = t.n2 >> 1;
    const unsigned low = static_cast<unsigned>(reinterpret_cast<uintptr_t>(t.g)) & 31u;
    const int vec = i + 8 > n ? 0 : low == 0 ? 2 : low == 16 ? 1 : 0;
    f2 g[4];
    if (t.n2 & 1) take<false>(static_cast<const bf16_t*>(t.g), i, n, vec != 0, g);
    else if (vec == 2) take<true>(static_cast<const float*>(t.g), i, n, true, g);
    else take<false>(static_cast<const float*>(t.g), i, n, vec != 0, g);
#pragma unroll
    for (int e = 0; e < 4; ++e) add_square(g[e], hi, lo, mul);
  }
  const float2 h2 = unpk(hi), l2 = unpk(lo);
  const float2 s = block_pair(add_pair(make_float2(h2.x, l2.x), make_float2(h2.y, l2.y)), s_sum);
  if (threadIdx.x == 0) tab.part[blockIdx.x] = s;
}

int64_t chunks_of(int64_t n) { return (n + kChunk - 1) / kChunk; }

// Blocks on an SM with 32-bit moments: two, though four fit (adapters of 52 M values
// with master copies and the clip 273 us against 276, 16 M bf16 values 55.7 against
// 58.4: fewer streams at once).  8-bit moments take what fits, five.
constexpr int kWideBlocks = 2;
template <typename PT, typename GT, bool MASTER, bool EIGHT, int MAX>
cudaError_t launch(const Table<MAX>& tab, cudaStream_t s) {
  static const int per = [] {
    int b = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
        &b, adamw_kernel<PT, GT, MASTER, EIGHT, MAX>, kThreads, 0);
    return e == cudaSuccess && b > 0 ? b : 1;
  }();
  const int blocks = std::min(tab.s.chunks, (EIGHT ? per : std::min(per, kWideBlocks)) * kSMs);
  return launch_pdl(adamw_kernel<PT, GT, MASTER, EIGHT, MAX>, dim3(blocks), dim3(kThreads), 0, s, tab);
}

int kind_of(const moe_adamw_tensor& t) {
  const int p = t.param_type == MOE_F32 ? 0 : t.master == nullptr ? 1 : 2;
  return (p * 2 + (t.grad_type == MOE_BF16 ? 1 : 0)) * 2 + (t.state_bits == 8 ? 1 : 0);
}
constexpr int kKinds = 12;

template <int MAX>
cudaError_t launch_kind(int kind, const Table<MAX>& tab, cudaStream_t s) {
  switch (kind) {
    case 0: return launch<float, float, false, false>(tab, s);
    case 1: return launch<float, float, false, true>(tab, s);
    case 2: return launch<float, bf16_t, false, false>(tab, s);
    case 3: return launch<float, bf16_t, false, true>(tab, s);
    case 4: return launch<bf16_t, float, false, false>(tab, s);
    case 5: return launch<bf16_t, float, false, true>(tab, s);
    case 6: return launch<bf16_t, bf16_t, false, false>(tab, s);
    case 7: return launch<bf16_t, bf16_t, false, true>(tab, s);
    case 8: return launch<bf16_t, float, true, false>(tab, s);
    case 9: return launch<bf16_t, float, true, true>(tab, s);
    case 10: return launch<bf16_t, bf16_t, true, false>(tab, s);
    default: return launch<bf16_t, bf16_t, true, true>(tab, s);
  }
}

// All tensors of one kind, up to MAX in a launch.
template <int MAX>
cudaError_t step_kind(int kind, const moe_adamw_tensor* ts, int n, const moe_adamw_hyper* h,
                      Consts& c, cudaStream_t s) {
  Table<MAX> tab;
  tab.c = c;
  tab.s.clear();
  const double b1t = 1.0 - std::pow(h->beta1, static_cast<double>(h->step));
  auto flush = [&]() -> cudaError_t {
    if (tab.s.n == 0) return cudaSuccess;
    tab.s.close();
    tab.c = c;
    const cudaError_t e = launch_kind<MAX>(kind, tab, s);
    c.norm_out = nullptr;  // written once
    tab.s.clear();
    return e;
  };
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor& q = ts[i];
    if (q.n == 0 || kind_of(q) != kind) continue;
    const int64_t ch = chunks_of(q.n);
    if (tab.s.full(ch)) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    Tensor& t = tab.t[tab.s.add(ch)];
    t.p = q.param; t.master = q.master; t.g = q.grad; t.m = q.m; t.v = q.v; t.sc = q.scales;
    t.n = q.n;
    const double lr = h->lr * static_cast<double>(q.lr_mult);
    t.keep = static_cast<float>(1.0 - lr * static_cast<double>(q.weight_decay));
    t.lr = static_cast<float>(lr / b1t);
    const uintptr_t wide = reinterpret_cast<uintptr_t>(q.param) | reinterpret_cast<uintptr_t>(q.master) |
                           reinterpret_cast<uintptr_t>(q.grad);
    const uintptr_t st = reinterpret_cast<uintptr_t>(q.m) | reinterpret_cast<uintptr_t>(q.v);
    t.vec = (wide & 15u) != 0 || (st & (q.state_bits == 8 ? 7u : 15u)) != 0      ? 0
            : (wide & 31u) != 0 || (q.state_bits == 32 && (st & 31u) != 0) ? 1
                                                                             : 2;
  }
  return flush();
}

template <int MAX>
cudaError_t norm_all(const moe_adamw_tensor* ts, int n, float2* part, int* nparts, cudaStream_t s) {
  NormTable<MAX> tab;
  tab.zero = -0.f;
  tab.s.clear();
  *nparts = 0;
  auto flush = [&]() -> cudaError_t {
    if (tab.s.n == 0) return cudaSuccess;
    tab.s.close();
    tab.part = part + *nparts;
    const int blocks = std::min(tab.s.chunks, kNormBlocks);
    *nparts += blocks;
    const cudaError_t e = launch_pdl(grad_norm_kernel<MAX>, dim3(blocks), dim3(kThreads), 0, s, tab);
    tab.s.clear();
    return e;
  };
  for (int i = 0; i < n; ++i) {
    if (ts[i].n == 0) continue;
    const int64_t ch = chunks_of(ts[i].n);
    if (tab.s.full(ch)) {
      const cudaError_t e = flush();
      if (e != cudaSuccess) return e;
    }
    tab.t[tab.s.add(ch)] = NormTensor{ts[i].grad, 2 * ts[i].n + (ts[i].grad_type == MOE_BF16 ? 1 : 0)};
  }
  return flush();
}

int bad(const char* msg) { return record_error(MOE_ERR_INVALID_ARG, msg); }

// Rows of partial sums: at most kNormBlocks for each norm launch.
size_t norm_rows(const moe_adamw_tensor* ts, int n) {
  int64_t launches = 1, in_launch = 0, chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (ts[i].n <= 0) continue;
    const int64_t ch = chunks_of(ts[i].n);
    const int most = n <= kNormFew ? kNormFew : n <= kNormSome ? kNormSome : kNormMany;
    if (in_launch == most || chunks + ch > (int64_t(1) << 30)) {
      ++launches;
      in_launch = chunks = 0;
    }
    ++in_launch;
    chunks += ch;
  }
  return static_cast<size_t>(launches) * kNormBlocks;
}

int check_tensor(const moe_adamw_tensor& t) {
  if (t.n < 0 || t.n > (int64_t(1) << 40)) return bad("a tensor's n is negative or above 2^40");
  if (t.param_type != MOE_F32 && t.param_type != MOE_BF16) return bad("param_type must be MOE_F32 or MOE_BF16");
  if (t.grad_type != MOE_F32 && t.grad_type != MOE_BF16) return bad("grad_type must be MOE_F32 or MOE_BF16");
  if (t.state_bits != 8 && t.state_bits != 32) return bad("state_bits must be 8 or 32");
  if (t.param_type == MOE_F32 && t.master != nullptr) return bad("an fp32 parameter has no master copy");
  if (!std::isfinite(t.weight_decay) || !std::isfinite(t.lr_mult) || t.weight_decay < 0.f || t.lr_mult < 0.f)
    return bad("weight_decay and lr_mult must be finite and not negative");
  if (t.n == 0) return MOE_OK;
  if (!t.param || !t.grad || !t.m || !t.v) return bad("NULL pointer in a tensor");
  if ((t.state_bits == 8) != (t.scales != nullptr)) return bad("scales go with 8-bit states");
  auto off = [](const void* p, unsigned size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; };
  const unsigned ss = t.state_bits == 8 ? 1 : 4;
  if (off(t.param, t.param_type == MOE_BF16 ? 2 : 4) || off(t.grad, t.grad_type == MOE_BF16 ? 2 : 4) ||
      off(t.master, 4) || off(t.m, ss) || off(t.v, ss))
    return bad("misaligned pointer in a tensor");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_adamw_workspace_size(const moe_adamw_tensor* tensors, int32_t n) {
  if (n < 0 || (n > 0 && tensors == nullptr)) return 0;
  return norm_rows(tensors, n) * sizeof(float2);
}

int moe_adamw_step(const moe_adamw_tensor* tensors, int32_t n, const moe_adamw_hyper* hyper,
                   float* grad_norm, void* ws, size_t ws_bytes, moe_stream_t stream) {
  NvtxScope nvtx("moe_adamw_step");
  if (n < 0 || (n > 0 && tensors == nullptr)) return bad("tensors is NULL or n negative");
  const moe_adamw_hyper* h = hyper;
  if (h == nullptr) return bad("hyper is NULL");
  if (!(h->lr >= 0.0) || !std::isfinite(h->lr)) return bad("lr must be finite and not negative");
  if (!(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0))
    return bad("betas must be in [0, 1)");
  if (!(h->eps >= 1e-30) || !(h->eps <= 1e30)) return bad("eps must be from 1e-30 to 1e30");
  if (!(h->max_norm >= 0.f) || !std::isfinite(h->max_norm)) return bad("max_norm must be finite and not negative");
  if (!std::isfinite(h->grad_scale)) return bad("grad_scale must be finite");
  if (h->step < 1) return bad("step counts from 1");
  if (h->skip_nonfinite != 0 && h->skip_nonfinite != 1) return bad("skip_nonfinite must be 0 or 1");
  bool work[kKinds] = {};
  int count[kKinds] = {};
  bool any = false;
  for (int i = 0; i < n; ++i) {
    const int rc = check_tensor(tensors[i]);
    if (rc) return rc;
    if (tensors[i].n == 0) continue;
    const int k = kind_of(tensors[i]);
    work[k] = any = true;
    ++count[k];
  }
  const bool need_norm = h->max_norm > 0.f || grad_norm != nullptr || h->skip_nonfinite;
  if (need_norm) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) & 15u)) return bad("ws NULL or misaligned");
    if (ws_bytes < moe_adamw_workspace_size(tensors, n))
      return record_error(MOE_ERR_WORKSPACE, "AdamW workspace too small");
    if (reinterpret_cast<uintptr_t>(grad_norm) & 3u) return bad("grad_norm misaligned");
  }
  if (!any) {
    if (grad_norm != nullptr) {
      const cudaError_t e = cudaMemsetAsync(grad_norm, 0, sizeof(float), stream);
      if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
    }
    return record_error(MOE_OK, "");
  }
  Consts c = {};
  c.zero = -0.f;
  c.b1 = static_cast<float>(h->beta1);
  c.c1 = static_cast<float>(1.0 - h->beta1);
  c.b2 = static_cast<float>(h->beta2);
  c.c2 = static_cast<float>(1.0 - h->beta2);
  c.correct = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(h->beta2, static_cast<double>(h->step))));
  c.eps = static_cast<float>(h->eps);
  c.grad_scale = h->grad_scale;
  c.max_norm = h->max_norm;
  c.dither = static_cast<uint32_t>(h->step) * kDitherT;
  c.skip = h->skip_nonfinite;
  c.norm_out = grad_norm;
  cudaError_t e = cudaSuccess;
  if (need_norm) {
    c.part = static_cast<const float2*>(ws);
    ProbeScope probe("grad_norm", stream);
    float2* part = static_cast<float2*>(ws);
    e = n <= kNormFew    ? norm_all<kNormFew>(tensors, n, part, &c.nparts, stream)
        : n <= kNormSome ? norm_all<kNormSome>(tensors, n, part, &c.nparts, stream)
                         : norm_all<kNormMany>(tensors, n, part, &c.nparts, stream);
  }
  ProbeScope probe("adamw", stream);
  for (int k = 0; k < kKinds && e == cudaSuccess; ++k) {
    if (!work[k]) continue;
    e = count[k] <= kFew    ? step_kind<kFew>(k, tensors, n, h, c, stream)
        : count[k] <= kSome ? step_kind<kSome>(k, tensors, n, h, c, stream)
                            : step_kind<kMany>(k, tensors, n, h, c, stream);
  }
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
