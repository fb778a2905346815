// Eight values of a row as one thread's share, widened to fp32 and held as four
// pairs: a pair is one 64-bit register for the packed fp32 operations
// (fma / mul / add of two values by one instruction).  Shared by the row-wise
// kernels.
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace moe {

constexpr int kSMs = 152;  // SMs of a GB300; grids of persistent kernels are multiples of it

struct bf16_t {  // storage type: a bf16 bit pattern
  uint16_t bits;
};

// ---- packed pairs -----------------------------------------------------------
struct f2 {
  uint64_t v;
};
__device__ __forceinline__ f2 pk(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 pk(float x) { return pk(x, x); }
__device__ __forceinline__ float2 unpk(f2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ float sum2(f2 a) {
  const float2 x = unpk(a);
  return x.x + x.y;
}

// ---- shares -------------------------------------------------------------------
// The registers that hold eight values as they are stored.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16_t> {
  uint4 v;
};
template <>
struct Raw8<float> {
  float4 a, b;
};

__device__ __forceinline__ void widen(const Raw8<bf16_t>& r, f2 (&f)[4]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = pk(bf16lo(w[i]), bf16hi(w[i]));
}
__device__ __forceinline__ void widen(const Raw8<float>& r, f2 (&f)[4]) {
  f[0] = pk(r.a.x, r.a.y); f[1] = pk(r.a.z, r.a.w);
  f[2] = pk(r.b.x, r.b.y); f[3] = pk(r.b.z, r.b.w);
}
__device__ __forceinline__ void narrow(const f2 (&f)[4], Raw8<bf16_t>& r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = unpk(f[i]);
    w[i] = pack_bf16x2(x.x, x.y);
  }
  r.v = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void narrow(const f2 (&f)[4], Raw8<float>& r) {
  const float2 a = unpk(f[0]), b = unpk(f[1]), c = unpk(f[2]), d = unpk(f[3]);
  r.a = make_float4(a.x, a.y, b.x, b.y);
  r.b = make_float4(c.x, c.y, d.x, d.y);
}

// Columns of a thread's share number `v` (a warp's 32 shares are consecutive):
// VEC: 8 v + e, moved as 16-byte words (rows 16-byte aligned, d a multiple of
// 8); else 256 (v / 32) + v % 32 + 32 e, so that a warp's element loads are
// consecutive whatever the row's alignment.
template <bool VEC>
__device__ __forceinline__ int col_of(int v, int e) {
  return VEC ? 8 * v + e : ((v >> 5) << 8) + (v & 31) + 32 * e;
}

// Loads read through the ordinary path (not the non-coherent one): callers
// may pass an output that aliases an input row for row.  Columns past d read 0.
template <bool VEC>
__device__ __forceinline__ void load8(const bf16_t* row, int v, int d, Raw8<bf16_t>& r) {
  r.v = make_uint4(0, 0, 0, 0);
  if (VEC) {
    if (8 * v < d) r.v = *(reinterpret_cast<const uint4*>(row) + v);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col_of<VEC>(v, e);
      w[e] = c < d ? row[c].bits : 0u;
    }
    r.v = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16),
                     w[6] | (w[7] << 16));
  }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int v, int d, Raw8<float>& r) {
  if (VEC) {
    r.a = r.b = make_float4(0.f, 0.f, 0.f, 0.f);
    if (8 * v < d) {
      r.a = *(reinterpret_cast<const float4*>(row) + 2 * v);
      r.b = *(reinterpret_cast<const float4*>(row) + 2 * v + 1);
    }
  } else {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col_of<VEC>(v, e);
      f[e] = c < d ? row[c] : 0.f;
    }
    r.a = make_float4(f[0], f[1], f[2], f[3]);
    r.b = make_float4(f[4], f[5], f[6], f[7]);
  }
}
// Eight floats at a 32-byte aligned address as one access: a warp's shares are
// then whole lines, where two 16-byte accesses each touch every line by half.
__device__ __forceinline__ void load8_wide(const float* p, Raw8<float>& r) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(r.a.x), "=f"(r.a.y), "=f"(r.a.z), "=f"(r.a.w), "=f"(r.b.x), "=f"(r.b.y),
                 "=f"(r.b.z), "=f"(r.b.w)
               : "l"(p));
}
__device__ __forceinline__ void store8_wide(float* p, const Raw8<float>& r) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(r.a.x),
               "f"(r.a.y), "f"(r.a.z), "f"(r.a.w), "f"(r.b.x), "f"(r.b.y), "f"(r.b.z), "f"(r.b.w)
               : "memory");
}

template <bool VEC>
__device__ __forceinline__ void store8(bf16_t* row, int v, int d, const Raw8<bf16_t>& r) {
  if (VEC) {
    if (8 * v < d) *(reinterpret_cast<uint4*>(row) + v) = r.v;
  } else {
    const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col_of<VEC>(v, e);
      if (c < d) row[c].bits = static_cast<uint16_t>(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void store8(float* row, int v, int d, const Raw8<float>& r) {
  if (VEC) {
    if (8 * v < d) {
      *(reinterpret_cast<float4*>(row) + 2 * v) = r.a;
      *(reinterpret_cast<float4*>(row) + 2 * v + 1) = r.b;
    }
  } else {
    const float f[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col_of<VEC>(v, e);
      if (c < d) row[c] = f[e];
    }
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void get8(const T* row, int v, int d, f2 (&f)[4]) {
  Raw8<T> r;
  load8<VEC>(row, v, d, r);
  widen(r, f);
}
template <typename T, bool VEC>
__device__ __forceinline__ void put8(T* row, int v, int d, const f2 (&f)[4]) {
  Raw8<T> r;
  narrow(f, r);
  store8<VEC>(row, v, d, r);
}

}  // namespace moe
