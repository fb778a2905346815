// Activation checkpoints in 8 bits.  A block of 32 consecutive values of a row
// shares the scale 2^e, e the least integer (>= -126) with max |x| <= 127 2^e:
//   code = rint(x 2^-e)  (int8),   scale byte = e + 127,   x' = code 2^e
// e is at most 121: above 127 2^121, within 0.8 % of the largest fp32 value, values
// count as that (64 2^122 would be infinite).
// 127 = 1.984375 * 2^6, so e is read off the largest value's bits: its exponent
// less 6, one more where its mantissa exceeds 0.984375 * 2^23 (a carry does it).
// Whole numbers and powers of two throughout: the one rounding is the code's.
// Power-of-two scales cost up to one of the codes' 7 bits, half a bit on average,
// against scales of any value; they make codes and results exact to state and
// restore, where a rounded quotient would move a code now and then.
//
// Memory bounds all three: 32768 x 1536 fp32 packed in 39 us, restored in 39 (both 0.95 of a
// copy's rate), restored with act in 58 (0.90); 16384 x 2880 bf16 packed in 27 (0.77) and
// restored in 23.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kCkptThreads = 256, kCkptWarps = kCkptThreads / 32;
constexpr int kSegCols = 256;  // columns of a warp's unit: 8 values, or every 32nd of 8, a lane
// Units whose loads are in flight at once: two when packing (four: 32768 x 1536 fp32 41 us
// against 39), and 16 bytes of codes a lane
// when unpacking fp32 and 32 bf16 (unpacking 16384 x 2880 into bf16: 23 us).
constexpr int kPackUnits = 2;
template <typename T>
constexpr int kUnpackUnits = 8 / sizeof(T);

// The bits of a block's largest |x| to its scale byte; 255 where it is not finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
  if (bits >= 0x7F800000u) return 255u;
  const int b = static_cast<int>((bits + 0x1FFFFu) >> 23) - 6;
  return static_cast<uint32_t>(b < 1 ? 1 : b);
}
// Blocks whose largest value is above 127 2^121: the scale stays and values are cut.
constexpr uint32_t kMaxByte = 248u;
constexpr float kMaxValue = 3.376239110640e38f;
__device__ __forceinline__ float cut(float x) { return fminf(fmaxf(x, -kMaxValue), kMaxValue); }
__device__ __forceinline__ f2 cut(f2 a) {
  const float2 x = unpk(a);
  return pk(cut(x.x), cut(x.y));
}
// 2^-e of a scale byte (any number for 255: the codes are set to 0 there).
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return __uint_as_float((254u - (byte == 255u ? 127u : byte)) << 23);
}
// 2^e, from 2^-127 on, which has no exponent byte of its own; NaN (infinity times 0) for
// 255.  By floating-point operations: odd rows restore 3 % faster than with masks and
// shifts (32768 x 1001 fp32 31.4 us, 32.5).
__device__ __forceinline__ float scale_of(uint32_t byte) {
  const float e = fmaxf(__uint_as_float(byte << 23), 0x1p-127f);
  return fmaf(e, 0.f, e);
}

// Rounding to the nearest integer by adding 1.5 * 2^23: the sum's last byte is the
// code (|x 2^-e| <= 127; the product is exact, so the fused sum rounds once).
constexpr float kRoundShift = 12582912.f;
__device__ __forceinline__ uint32_t four_codes(f2 a, f2 b, f2 s) {
  const float2 u = unpk(fma2(a, s, pk(kRoundShift))), v = unpk(fma2(b, s, pk(kRoundShift)));
  const uint32_t lo = __byte_perm(__float_as_uint(u.x), __float_as_uint(u.y), 0x0040);
  const uint32_t hi = __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }
// The bits of a share's largest |x|, as an fp32 value has them.
__device__ __forceinline__ uint32_t share_max(const Raw8<bf16_t>& r) {
  const uint32_t m = __vmaxu2(__vmaxu2(r.v.x & 0x7FFF7FFFu, r.v.y & 0x7FFF7FFFu),
                              __vmaxu2(r.v.z & 0x7FFF7FFFu, r.v.w & 0x7FFF7FFFu));
  return max(m & 0xFFFF0000u, m << 16);
}
__device__ __forceinline__ uint32_t share_max(const Raw8<float>& r) {
  return max(max(max(abs_bits(r.a.x), abs_bits(r.a.y)), max(abs_bits(r.a.z), abs_bits(r.a.w))),
             max(max(abs_bits(r.b.x), abs_bits(r.b.y)), max(abs_bits(r.b.z), abs_bits(r.b.w))));
}
// Codes to values: a byte b, its sign bit flipped, as the last byte of 2^23 is
// 2^23 + 128 + b.
__device__ __forceinline__ void four_values(uint32_t codes, f2 scale, f2& a, f2& b) {
  const uint32_t u = codes ^ 0x80808080u;
  const f2 shift = pk(-8388736.f);
  a = mul2(add2(pk(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7540)),
                   __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7541))), shift), scale);
  b = mul2(add2(pk(__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7542)),
                   __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7543))), shift), scale);
}

// Where unit u's columns lie: of row `row` from column `col` on, `segs` units to a row.
// FLAT: one row, without a division.
template <bool FLAT>
__device__ __forceinline__ void unit_place(int64_t u, int64_t segs, int64_t& row, int64_t& col) {
  if (FLAT) row = 0;
  else if ((u >> 32) == 0) row = static_cast<uint32_t>(u) / static_cast<uint32_t>(segs);
  else row = u / segs;
  col = (FLAT ? u : u - row * segs) * kSegCols;
}

__device__ __forceinline__ void load_share(const bf16_t* p, Raw8<bf16_t>& r) {
  r.v = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void load_share(const float* p, Raw8<float>& r) { load8_wide(p, r); }
__device__ __forceinline__ void store_share(bf16_t* p, const Raw8<bf16_t>& r) {
  *reinterpret_cast<uint4*>(p) = r.v;
}
__device__ __forceinline__ void store_share(float* p, const Raw8<float>& r) { store8_wide(p, r); }
__device__ __forceinline__ float widen1(bf16_t x) { return __uint_as_float(uint32_t(x.bits) << 16); }
__device__ __forceinline__ float widen1(float x) { return x; }
__device__ __forceinline__ void narrow1(float x, float* p) { *p = x; }
__device__ __forceinline__ void narrow1(float x, bf16_t* p) {
  p->bits = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
}

// How the values are reached.  kFlat: the rows have no gaps between blocks (C a multiple
// of 32) and count as one row of R C columns, kRows: they do not; in both a lane has 8
// consecutive values, four lanes a block.  kSingle: a lane has every 32nd value and a
// warp's 32 lanes are a block, so that loads of any alignment and width cover whole
// sectors.
enum { kFlat = 0, kRows = 1, kSingle = 2 };

// C columns a row, nb blocks a row.  A block's warps have neighbouring units.
template <typename T, int HOW>
__global__ void __launch_bounds__(kCkptThreads) ckpt_pack_kernel(const T* __restrict__ x, int64_t R,
                                                                int64_t C, int64_t nb,
                                                                int8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales) {
  constexpr bool FLAT = HOW == kFlat;
  const int lane = threadIdx.x & 31;
  const int64_t segs = (C + kSegCols - 1) / kSegCols, units = R * segs;
  pdl_wait();
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kCkptWarps * kPackUnits + (threadIdx.x >> 5);
  if (HOW != kSingle) {
    Raw8<T> raw[kPackUnits];
    int64_t at[kPackUnits];  // of the lane's values, -1: none
    int64_t block[kPackUnits];
#pragma unroll
    for (int i = 0; i < kPackUnits; ++i) {
      // lanes past the end load the first values, so that no load waits for a branch
      const int64_t u = u0 + i * kCkptWarps;
      int64_t row, col;
      unit_place<FLAT>(u, segs, row, col);
      col += 8 * lane;
      const bool ok = u < units && col < C;
      at[i] = ok ? row * C + col : -1;
      block[i] = row * nb + col / MOE_CKPT_BLOCK;
      load_share(x + (ok ? at[i] : 0), raw[i]);
    }
#pragma unroll
    for (int i = 0; i < kPackUnits; ++i) {
      if (u0 + i * kCkptWarps >= units) break;
      uint32_t big = at[i] >= 0 ? share_max(raw[i]) : 0u;
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      f2 f[4];
      widen(raw[i], f);
      uint32_t byte = scale_byte(big);
      if (byte == kMaxByte + 1) {
        byte = kMaxByte;
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = cut(f[e]);
      }
      const f2 s = pk(inverse_scale(byte));
      uint2 q = make_uint2(four_codes(f[0], f[1], s), four_codes(f[2], f[3], s));
      if (byte == 255u) q = make_uint2(0u, 0u);
      if (at[i] >= 0) {
        *reinterpret_cast<uint2*>(codes + at[i]) = q;
        if ((lane & 3) == 0) scales[block[i]] = static_cast<uint8_t>(byte);
      }
    }
  } else {
    float f[kPackUnits][8];
    int64_t at[kPackUnits], block[kPackUnits];  // of the lane's first value, of the unit's first block
    int left[kPackUnits];                       // columns from the lane's first value to the row's end
#pragma unroll
    for (int i = 0; i < kPackUnits; ++i) {
      int64_t row, col;
      unit_place<false>(u0 + i * kCkptWarps, segs, row, col);
      at[i] = row * C + col + lane;
      block[i] = row * nb + col / MOE_CKPT_BLOCK;
      left[i] = u0 + i * kCkptWarps < units ? static_cast<int>(C - col) - lane : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = 32 * e < left[i] ? widen1(x[at[i] + 32 * e]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kPackUnits; ++i) {
      // the 8 blocks' largest, that of block lane / 4 in each lane: in each exchange a lane
      // hands half of its blocks to another.  (32768 x 1001: 41 us, with a reduction over
      // the warp for each block, and its scale in every lane, 52.)
      uint32_t big[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) big[e] = abs_bits(f[i][e]);
#pragma unroll
      for (int n = 4; n > 0; n >>= 1) {
        const bool upper = (lane & 4 * n) != 0;
#pragma unroll
        for (int e = 0; e < n; ++e) {
          const uint32_t give = upper ? big[e] : big[e + n], keep = upper ? big[e + n] : big[e];
          big[e] = max(keep, __shfl_xor_sync(0xffffffffu, give, 4 * n));
        }
      }
      big[0] = max(big[0], __shfl_xor_sync(0xffffffffu, big[0], 2));
      big[0] = max(big[0], __shfl_xor_sync(0xffffffffu, big[0], 1));
      uint32_t byte = scale_byte(big[0]);
      if (byte == kMaxByte + 1) byte = kMaxByte;
      const float inverse = byte == 255u ? 0.f : inverse_scale(byte);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = __shfl_sync(0xffffffffu, inverse, 4 * e);
        const uint32_t q = __float_as_uint(fmaf(cut(f[i][e]), s, kRoundShift));
        if (32 * e < left[i]) codes[at[i] + 32 * e] = static_cast<int8_t>(s == 0.f ? 0u : q & 0xFFu);
      }
      if ((lane & 3) == 0 && 7 * lane < left[i]) scales[block[i] + lane / 4] = static_cast<uint8_t>(byte);
    }
  }
}

template <typename T, int HOW>
__global__ void __launch_bounds__(kCkptThreads) ckpt_unpack_kernel(const int8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales,
                                                                  int64_t R, int64_t C, int64_t nb,
                                                                  T* __restrict__ x) {
  constexpr int kUnits = kUnpackUnits<T>;
  constexpr bool FLAT = HOW == kFlat;
  const int lane = threadIdx.x & 31;
  const int64_t segs = (C + kSegCols - 1) / kSegCols, units = R * segs;
  pdl_wait();
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * kCkptWarps * kUnits + (threadIdx.x >> 5);
  if (HOW != kSingle) {
    uint2 q[kUnits];
    uint32_t byte[kUnits];
    int64_t at[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      // lanes past the end load the first values, so that no load waits for a branch
      const int64_t u = u0 + i * kCkptWarps;
      int64_t row, col;
      unit_place<FLAT>(u, segs, row, col);
      col += 8 * lane;
      const bool ok = u < units && col < C;
      at[i] = ok ? row * C + col : -1;
      q[i] = __ldg(reinterpret_cast<const uint2*>(codes + (ok ? at[i] : 0)));
      byte[i] = __ldg(scales + (ok ? row * nb + col / MOE_CKPT_BLOCK : 0));
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (at[i] < 0) continue;
      const f2 s = pk(scale_of(byte[i]));
      f2 f[4];
      four_values(q[i].x, s, f[0], f[1]);
      four_values(q[i].y, s, f[2], f[3]);
      Raw8<T> raw;
      narrow(f, raw);
      store_share(x + at[i], raw);
    }
  } else {
    int q[kUnits][8];
    uint32_t byte[kUnits];  // the scale of block `lane`
    int64_t at[kUnits];
    int left[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      int64_t row, col;
      unit_place<false>(u0 + i * kCkptWarps, segs, row, col);
      at[i] = row * C + col + lane;
      left[i] = u0 + i * kCkptWarps < units ? static_cast<int>(C - col) - lane : 0;
      byte[i] = lane < 8 && 31 * lane < left[i] ? __ldg(scales + row * nb + col / MOE_CKPT_BLOCK + lane) : 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e) q[i][e] = 32 * e < left[i] ? __ldg(codes + at[i] + 32 * e) : 0;
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const float mine = scale_of(byte[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // fp32: a scale after its byte's exchange (32768 x 1001: 31.4 us, 32.7 as for bf16, whose
        // more units in flight are better off with one a lane: 26.8 us, 27.6)
        const float scale = sizeof(T) == 4 ? scale_of(__shfl_sync(0xffffffffu, byte[i], e))
                                           : __shfl_sync(0xffffffffu, mine, e);
        if (32 * e < left[i]) narrow1(static_cast<float>(q[i][e]) * scale, x + at[i] + 32 * e);
      }
    }
  }
}

// A thread takes 8 features: half of a chunk's gates and their ups.  `per` such
// items to a row (hs / 16), of which those past f have no act.  The writes bound it, and
// one item a thread, so more blocks, is faster than two or four (32768 rows of 768
// features 60, 64, 70 us).  wide: h is 32-byte aligned.
__global__ void __launch_bounds__(kCkptThreads) ckpt_unpack_swiglu_kernel(
    const int8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t items, unsigned per, int f,
    const int32_t* __restrict__ sorted_src, const float* __restrict__ topk_w, int P, int k, int K,
    float* __restrict__ h, bool wide, uint16_t* __restrict__ act, int64_t pair) {
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kCkptThreads;
  const int64_t row0 = base / per;
  const unsigned at = static_cast<unsigned>(base - row0 * per) + threadIdx.x;
  const unsigned r = at / per;
  const int half = static_cast<int>(at - r * per);
  const int64_t p = row0 + r;
  pdl_wait();
  if (base + threadIdx.x >= items) return;
  const int src = __ldg(sorted_src + p);
  if (src < 0 || src >= P) return;  // P = T K
  const int64_t first = p * (16 * static_cast<int64_t>(per)) + 32 * (half >> 1) + 8 * (half & 1);
  const uint2 gate = __ldg(reinterpret_cast<const uint2*>(codes + first));
  const uint2 up = __ldg(reinterpret_cast<const uint2*>(codes + first + 16));
  const f2 s = pk(scale_of(__ldg(scales + p * (per >> 1) + (half >> 1))));
  const int t = src / K, j = src - t * K;
  const float w = j < k ? __ldg(topk_w + static_cast<int64_t>(t) * k + j) : 1.f;
  f2 g[4], u[4];
  four_values(gate.x, s, g[0], g[1]);
  four_values(gate.y, s, g[2], g[3]);
  four_values(up.x, s, u[0], u[1]);
  four_values(up.y, s, u[2], u[3]);
  Raw8<float> raw[2];
  narrow(g, raw[0]);
  narrow(u, raw[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float* to = h + first + 16 * i;
    if (wide) {
      store8_wide(to, raw[i]);
    } else {
      *reinterpret_cast<float4*>(to) = raw[i].a;
      *reinterpret_cast<float4*>(to + 4) = raw[i].b;
    }
  }
  if (8 * half >= f) return;
  uint32_t hi[4], lo[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 a = unpk(g[e]), b = unpk(u[e]);
    const float x = w * (a.x / (1.f + expf(-a.x))) * b.x;
    const float y = w * (a.y / (1.f + expf(-a.y))) * b.y;
    hi[e] = pack_bf16x2(x, y);
    lo[e] = pack_bf16x2(x - bf16lo(hi[e]), y - bf16hi(hi[e]));
  }
  uint16_t* out = act + p * f + 8 * half;
  *reinterpret_cast<uint4*>(out) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  *reinterpret_cast<uint4*>(out + pair) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
}

int bad(const char* msg) { return record_error(MOE_ERR_INVALID_ARG, msg); }
bool misaligned(const void* p, unsigned size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; }

int check_rows(const void* x, int32_t x_type, int32_t R, int32_t C, const void* codes, const void* scales) {
  if (R < 0 || C <= 0) return bad("R must not be negative, C must be positive");
  if (x_type != MOE_F32 && x_type != MOE_BF16) return bad("x_type must be MOE_F32 or MOE_BF16");
  if (R == 0) return MOE_OK;
  if (!x || !codes || !scales) return bad("NULL pointer");
  if (misaligned(x, x_type == MOE_BF16 ? 2 : 4)) return bad("x is misaligned");
  return MOE_OK;
}

struct CkptShape {
  int64_t R, C, nb, blocks;
  int how;
};
CkptShape ckpt_shape(const void* x, int32_t x_type, int64_t R, int64_t C, const void* codes, int at_once) {
  CkptShape q{R, C, (C + MOE_CKPT_BLOCK - 1) / MOE_CKPT_BLOCK, 0, kRows};
  if (C % 8 != 0 || misaligned(x, x_type == MOE_BF16 ? 16 : 32) || misaligned(codes, 8)) q.how = kSingle;
  else if (C % MOE_CKPT_BLOCK == 0) q = CkptShape{1, R * C, R * q.nb, 0, kFlat};
  const int64_t units = q.R * ((q.C + kSegCols - 1) / kSegCols), per = kCkptWarps * at_once;
  q.blocks = (units + per - 1) / per;
  return q;
}

template <typename T>
cudaError_t pack(const void* x, int type, int64_t R, int64_t C, int8_t* codes, uint8_t* scales, cudaStream_t s) {
  const CkptShape q = ckpt_shape(x, type, R, C, codes, kPackUnits);
  if (q.blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(q.how == kFlat   ? ckpt_pack_kernel<T, kFlat>
                    : q.how == kRows ? ckpt_pack_kernel<T, kRows>
                                     : ckpt_pack_kernel<T, kSingle>,
                    dim3(static_cast<unsigned>(q.blocks)), dim3(kCkptThreads), 0, s, static_cast<const T*>(x), q.R,
                    q.C, q.nb, codes, scales);
}
template <typename T>
cudaError_t unpack(const int8_t* codes, const uint8_t* scales, int64_t R, int64_t C, void* x, int type,
                   cudaStream_t s) {
  const CkptShape q = ckpt_shape(x, type, R, C, codes, kUnpackUnits<T>);
  if (q.blocks > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  return launch_pdl(q.how == kFlat   ? ckpt_unpack_kernel<T, kFlat>
                    : q.how == kRows ? ckpt_unpack_kernel<T, kRows>
                                     : ckpt_unpack_kernel<T, kSingle>,
                    dim3(static_cast<unsigned>(q.blocks)), dim3(kCkptThreads), 0, s, codes, scales, q.R, q.C, q.nb,
                    static_cast<T*>(x));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

int moe_ckpt_pack(const void* x, int32_t x_type, int32_t R, int32_t C, int8_t* codes, uint8_t* scales,
                  moe_stream_t stream) {
  NvtxScope nvtx("moe_ckpt_pack");
  const int rc = check_rows(x, x_type, R, C, codes, scales);
  if (rc) return rc;
  if (R == 0) return record_error(MOE_OK, "");
  ProbeScope probe("ckpt_pack", stream);
  const cudaError_t e = x_type == MOE_BF16 ? pack<bf16_t>(x, x_type, R, C, codes, scales, stream)
                                           : pack<float>(x, x_type, R, C, codes, scales, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

int moe_ckpt_unpack(const int8_t* codes, const uint8_t* scales, int32_t R, int32_t C, void* x,
                    int32_t x_type, moe_stream_t stream) {
  NvtxScope nvtx("moe_ckpt_unpack");
  const int rc = check_rows(x, x_type, R, C, codes, scales);
  if (rc) return rc;
  if (R == 0) return record_error(MOE_OK, "");
  ProbeScope probe("ckpt_unpack", stream);
  const cudaError_t e = x_type == MOE_BF16 ? unpack<bf16_t>(codes, scales, R, C, x, x_type, stream)
                                           : unpack<float>(codes, scales, R, C, x, x_type, stream);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

int moe_ckpt_unpack_swiglu(const int8_t* codes, const uint8_t* scales, int32_t P, int32_t f,
                           const int32_t* sorted_src, const float* topk_w, int32_t k,
                           int32_t shared_expert, float* h, moe_bf16* act, moe_stream_t stream) {
  NvtxScope nvtx("moe_ckpt_unpack_swiglu");
  if (P < 0 || f <= 0 || f % 8 != 0) return bad("P must not be negative, f a positive multiple of 8");
  if (k <= 0 || k > 32 || (shared_expert != 0 && shared_expert != 1)) return bad("bad k or shared_expert");
  if (P % (k + shared_expert) != 0) return bad("P must be a multiple of k + shared_expert");
  if (P == 0) return record_error(MOE_OK, "");
  if (!codes || !scales || !sorted_src || !topk_w || !h || !act) return bad("NULL pointer");
  if (misaligned(codes, 8) || misaligned(sorted_src, 4) || misaligned(topk_w, 4) || misaligned(h, 16) ||
      misaligned(act, 16))
    return bad("misaligned pointer");
  const unsigned per = 2 * static_cast<unsigned>((static_cast<int64_t>(f) + 15) / 16);
  const int64_t items = static_cast<int64_t>(P) * per, blocks = (items + kCkptThreads - 1) / kCkptThreads;
  if (blocks > 0x7FFFFFFF) return record_error(MOE_ERR_UNSUPPORTED, "P x f is too large");
  ProbeScope probe("ckpt_unpack_swiglu", stream);
  const cudaError_t e = launch_pdl(ckpt_unpack_swiglu_kernel, dim3(static_cast<unsigned>(blocks)),
                                   dim3(kCkptThreads), 0, stream, codes, scales, items, per, f, sorted_src,
                                   topk_w, P, k, k + shared_expert, h, !misaligned(h, 32), act,
                                   static_cast<int64_t>(P) * f);
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
