// Eight consecutive (or lane-strided) values of a row as one thread's share,
// widened to fp32.  Shared by the row-wise kernels (norm.cu).
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace moe {

constexpr int kSMs = 152;  // SMs of a GB300; grids of persistent kernels are multiples of it

struct bf16_t {  // storage type tag: 16-bit pattern
  uint16_t bits;
};

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

__device__ __forceinline__ void widen(const Raw8<bf16_t>& r, float (&f)[8]) {
  const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ void widen(const Raw8<float>& r, float (&f)[8]) {
  f[0] = r.a.x; f[1] = r.a.y; f[2] = r.a.z; f[3] = r.a.w;
  f[4] = r.b.x; f[5] = r.b.y; f[6] = r.b.z; f[7] = r.b.w;
}
__device__ __forceinline__ void narrow(const float (&f)[8], Raw8<bf16_t>& r) {
  r.v = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                   pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void narrow(const float (&f)[8], Raw8<float>& r) {
  r.a = make_float4(f[0], f[1], f[2], f[3]);
  r.b = make_float4(f[4], f[5], f[6], f[7]);
}

// Columns of a thread's share number `v` (a warp's 32 shares are consecutive):
// VEC: 8 v + e, moved as 16-byte words (rows 16-byte aligned, d a multiple of
// 8); else 256 (v / 32) + v % 32 + 32 e, so that a warp's element loads are
// consecutive whatever the row's alignment.
template <bool VEC>
__device__ __forceinline__ int col_of(int v, int e) {
  return VEC ? 8 * v + e : ((v >> 5) << 8) + (v & 31) + 32 * e;
}
// Whether any column of share v lies in the row.
template <bool VEC>
__device__ __forceinline__ bool any_col(int v, int d) {
  return col_of<VEC>(v, 0) < d;
}

// Loads read through the ordinary path (not the non-coherent one): callers
// may pass an output that aliases an input row for row.
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
    narrow(f, r);
  }
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
    float f[8];
    widen(r, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = col_of<VEC>(v, e);
      if (c < d) row[c] = f[e];
    }
  }
}
// Eight fp32 values of a per-column vector (norm weights, channel gate).  Such
// a vector is read element by element unless VEC (then 16-byte aligned).
template <bool VEC>
__device__ __forceinline__ void load8f(const float* p, int v, int d, float (&f)[8]) {
  Raw8<float> r;
  load8<VEC>(p, v, d, r);
  widen(r, f);
}
template <typename T, bool VEC>
__device__ __forceinline__ void put8(T* row, int v, int d, const float (&f)[8]) {
  Raw8<T> r;
  narrow(f, r);
  store8<VEC>(row, v, d, r);
}

}  // namespace moe
