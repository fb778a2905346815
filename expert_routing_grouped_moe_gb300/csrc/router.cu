// The router's two losses and the gradient of its logits.
//   P = softmax(l),  lse = log sum_e exp l,  f_e = counts_e / (T k)
//   aux = E sum_e f_e mean_t P_te            z = mean_t lse_t^2
//   dl_te = c_aux E/T P_te (f_e - sum_e' f_e' P_te') + 2 c_z/T lse_t P_te
//         + sum_{j: ids_tj = e} w_tj (dw_tj - sum_i w_ti dw_ti)
// A row is held by LPR lanes (a power of two), NV vectors of 4 logits each.  A
// row whose logits are all -inf has P = 0, adds nothing to either loss and
// gets a zero gradient; its lse is -inf.
// Each pass reads the logits once, as float4 where rows allow.  1,048,576 x 128:
// losses 92 us, 5.9 TB/s (0.87 of a plain copy's rate), gradient 195 us, 6.0 TB/s
// (0.89; 187 us without the second sum of a row); the loads' latency bounds them
// (16 logits a lane in flight).  4096 x 128: losses
// 5.8 us, of which the two launches and the last sum are 4.
#include <algorithm>
#include <cstdint>

#include "../../include/moe_gb300.h"
#include "internal.h"
#include "ptx.cuh"
#include "rowvec.cuh"

namespace moe {
namespace {

constexpr int kRouterThreads = 256;
constexpr int kRouterWarps = kRouterThreads / 32;
// Blocks of the forward, which also bound the rows of partial sums: four for
// each SM.
constexpr int kRouterBlocks = 4 * kSMs;
// The losses in one launch: one cluster of up to 8 blocks of 1024 threads, for up
// to 131,072 logits (within a graph 64 x 60: 3.4 us, 5.5 with two launches;
// 1024 x 128: 5.0 and 5.8; 4096 x 128: 8.2 and 5.8).
constexpr int kOneThreads = 1024, kOneBlocks = 8, kOneMaxE = 256;
constexpr int64_t kOneMaxLogits = int64_t(1) << 17;

// Rows that 8 lanes load before they work on the first: 16 logits a lane in flight.
__host__ __device__ constexpr int rows_at_once(int lpr, int nv) { return lpr == 8 ? 4 / nv : 1; }

template <bool VEC, int LPR>
__device__ __forceinline__ int ecol(int sub, int i, int e) {
  return VEC ? 4 * (sub + LPR * i) + e : sub + LPR * (4 * i + e);
}
template <bool VEC, int LPR, int NV>
__device__ __forceinline__ void load_row(const float* row, int sub, int E, float fill,
                                         float (&l)[NV][4]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if (VEC) {
      float4 q = make_float4(fill, fill, fill, fill);
      if (ecol<VEC, LPR>(sub, i, 0) < E) q = __ldg(reinterpret_cast<const float4*>(row) + sub + LPR * i);
      l[i][0] = q.x; l[i][1] = q.y; l[i][2] = q.z; l[i][3] = q.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = ecol<VEC, LPR>(sub, i, e);
        l[i][e] = c < E ? __ldg(row + c) : fill;
      }
    }
  }
}
template <int LPR>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Two sums at once: after the first exchange each half of the lanes carries one.
template <int LPR>
__device__ __forceinline__ void lanes_sums(float& a, float& b) {
  if (LPR < 4) {
    a = lanes_sum<LPR>(a);
    b = lanes_sum<LPR>(b);
    return;
  }
  const bool up = threadIdx.x & (LPR / 2);
  float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, LPR / 2);
#pragma unroll
  for (int o = LPR / 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const float w = __shfl_xor_sync(0xffffffffu, v, LPR / 2);
  a = up ? w : v;
  b = up ? v : w;
}
template <int LPR>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

struct LossEnd {           // what the last sum writes
  const int32_t* counts;
  int k;
  float *losses, *pmean;
};

// pmean of column e from its sum over all rows (e = E: the z loss); returns the
// column's share of the load-balancing sum.
__device__ __forceinline__ float end_column(const LossEnd& o, int e, int E, float t, float inv_T) {
  t *= inv_T;
  if (e == E) {
    o.losses[1] = t;
    return 0.f;
  }
  o.pmean[e] = t;
  return static_cast<float>(o.counts[e]) * t;
}
__device__ __forceinline__ void end_aux(const LossEnd& o, float aux, int T, int E) {
  o.losses[0] = aux * (static_cast<float>(E) / (static_cast<float>(T) * static_cast<float>(o.k)));
}
// Sum over a block of 1024 threads, in thread 0 (all of warp 0); s_aux: 32 floats.
__device__ __forceinline__ float block_aux(float aux, float* s_aux) {
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) aux += __shfl_xor_sync(0xffffffffu, aux, i);
  if ((threadIdx.x & 31) == 0) s_aux[threadIdx.x >> 5] = aux;
  __syncthreads();
  if (threadIdx.x < 32) {
    aux = s_aux[threadIdx.x];
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) aux += __shfl_xor_sync(0xffffffffu, aux, i);
  }
  return aux;
}
// A shared variable of the cluster's block q.
__device__ __forceinline__ float cluster_float(const float* p, unsigned q) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(p), q)) : "memory");
  return v;
}

// part: [gridDim.x][ld]: sums of P over the block's rows, then of lse^2, then zeros.
// ONE: the whole grid is one cluster, whose first block adds the blocks' sums up
// out of their shared memory and writes the result: no second kernel.
template <bool VEC, int LPR, int NV, bool ONE>
__global__ void __launch_bounds__(ONE ? kOneThreads : kRouterThreads) router_loss_kernel(
    const float* __restrict__ logits, int T, int E, float* __restrict__ lse, float* __restrict__ part,
    int ld, const LossEnd end) {
  constexpr int kRouterWarps = (ONE ? kOneThreads : kRouterThreads) / 32, U = rows_at_once(LPR, NV);
  extern __shared__ float s_acc[];  // [kRouterWarps][ld]
  constexpr int RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR, r = lane / LPR;
  float acc[NV][4], zacc = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  pdl_wait();
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouterWarps * RPW * U;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouterWarps + warp) * RPW * U; t0 < T;
       t0 += step) {
    float rows[U][NV][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * RPW + r;
      load_row<VEC, LPR, NV>(logits + (t < T ? t * E : 0), sub, t < T ? E : 0, -INFINITY, rows[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * RPW + r;
      float(&l)[NV][4] = rows[u];
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) m = fmaxf(m, l[i][e]);
      m = lanes_max<LPR>(m);
      const float m0 = m == -INFINITY ? 0.f : m;  // an empty row: every term 0
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[i][e] = __expf(l[i][e] - m0);
          s += l[i][e];
        }
      s = lanes_sum<LPR>(s);
      const bool some = s != 0.f;  // also where s is NaN
      const float inv = some ? 1.f / s : 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(l[i][e], inv, acc[i][e]);
      const float ls = some ? m0 + logf(s) : -INFINITY;
      if (t < T && sub == 0) {
        lse[t] = ls;
        if (some) zacc = fmaf(ls, ls, zacc);
      }
    }
  }
  // over the row groups of a warp, then over the warps
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
    zacc += __shfl_xor_sync(0xffffffffu, zacc, o);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] += __shfl_xor_sync(0xffffffffu, acc[i][e], o);
  }
  if (r == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = ecol<VEC, LPR>(sub, i, e);
        if (c < E) s_acc[warp * ld + c] = acc[i][e];
      }
    if (sub == 0) s_acc[warp * ld + E] = zacc;
  }
  __syncthreads();
  if (!ONE) {
    for (int c = threadIdx.x; c < ld; c += kRouterThreads) {
      float v = 0.f;
      if (c <= E) {
#pragma unroll
        for (int w = 0; w < kRouterWarps; ++w) v += s_acc[w * ld + c];
      }
      part[static_cast<int64_t>(blockIdx.x) * ld + c] = v;
    }
    return;
  }
  __shared__ float s_sum[kOneMaxE + 1], s_aux[32];
  if (threadIdx.x <= E) {
    float v = 0.f;
#pragma unroll 8
    for (int w = 0; w < kRouterWarps; ++w) v += s_acc[w * ld + threadIdx.x];
    s_sum[threadIdx.x] = v;
  }
  cluster_sync();
  if (cluster_ctarank() == 0) {
    float aux = 0.f;
    if (threadIdx.x <= E) {
      float t = 0.f;
      for (unsigned q = 0; q < gridDim.x; ++q) t += cluster_float(&s_sum[threadIdx.x], q);
      aux = end_column(end, threadIdx.x, E, t, 1.f / static_cast<float>(T));
    }
    aux = block_aux(aux, s_aux);
    if (threadIdx.x == 0) end_aux(end, aux, T, E);
  }
  cluster_sync();  // no block leaves while its sums are read
}

// One cluster: pmean, then losses[0] = aux, losses[1] = z, from P rows of partials
// of `ld` floats (E sums of P, the sum of lse^2, zeros up to a multiple of 4).
// Each block takes a share of the columns; each of its threads adds every G-th
// row of one vector of 4 columns, all loads independent; then the G sums of a
// column are added in order, and the blocks' shares of aux by the first block.
constexpr int kFinalThreads = 1024, kFinalBlocks = 8;
__global__ void __launch_bounds__(kFinalThreads) router_loss_final_kernel(
    const float* __restrict__ part, int P, int ld, int T, int E, const LossEnd end) {
  __shared__ float4 s_col[kFinalThreads];
  __shared__ float s_aux[32], s_share;
  const int nv = ld / 4, per = (nv + gridDim.x - 1) / gridDim.x;  // vectors in all; of this block
  const int v0 = blockIdx.x * per, mine = nv - v0 < per ? nv - v0 : per;
  const int G = kFinalThreads / per;
  const int g = threadIdx.x / per, c = threadIdx.x - g * per;
  pdl_wait();
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (g < G && c < mine) {
    const float4* col = reinterpret_cast<const float4*>(part) + v0 + c;
#pragma unroll 8
    for (int b = g; b < P; b += G) {
      const float4 q = col[static_cast<int64_t>(b) * nv];
      v.x += q.x; v.y += q.y; v.z += q.z; v.w += q.w;
    }
  }
  s_col[threadIdx.x] = v;
  __syncthreads();
  // a warp adds up a column: lanes every 32nd of the G sums, then the lanes
  float aux = 0.f;
  for (int q = threadIdx.x >> 5; q < 4 * mine; q += kFinalThreads / 32) {
    const int e = 4 * v0 + q;
    float t = 0.f;
    for (int r = threadIdx.x & 31; r < G; r += 32)
      t += reinterpret_cast<const float*>(s_col)[r * 4 * per + q];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0 && e <= E) aux += end_column(end, e, E, t, 1.f / static_cast<float>(T));
  }
  aux = block_aux(aux, s_aux);
  if (threadIdx.x == 0) s_share = aux;
  cluster_sync();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    aux = 0.f;
    for (unsigned q = 0; q < gridDim.x; ++q) aux += cluster_float(&s_share, q);
    end_aux(end, aux, T, E);
  }
  cluster_sync();  // no block leaves while its share is read
}

// The gradient rows of a warp pass through shared memory for the top-k terms:
// lane `sub` of a row adds the terms of slots sub, sub + LPR, ...  Slots of one
// row name different experts (then no two lanes meet); each slot first writes
// its number where its term goes and reads it back, and where that shows an
// expert named twice the terms are added slot by slot instead.
template <bool VEC, int LPR, int NV>
__global__ void __launch_bounds__(kRouterThreads) router_bwd_kernel(
    const float* __restrict__ logits, const float* __restrict__ lse,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ ids,
    const float* __restrict__ w, const float* __restrict__ dw, int T, int E, int k, float c_aux,
    float c_z, float inv_Tk, float* __restrict__ dlogits, int* status) {
  extern __shared__ float4 s_rows[];  // [kRouterWarps][RPW][4 LPR NV]
  constexpr int RPW = 32 / LPR, LD = 4 * LPR * NV, U = rows_at_once(LPR, NV);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % LPR, r = lane / LPR;
  float* s_row = reinterpret_cast<float*>(s_rows) + (warp * RPW + r) * LD;
  pdl_wait();
  float f[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int c = ecol<VEC, LPR>(sub, i, e);
      f[i][e] = counts != nullptr && c < E ? static_cast<float>(__ldg(counts + c)) * inv_Tk : 0.f;
    }
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRouterWarps * RPW * U;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kRouterWarps + warp) * RPW * U; t0 < T;
       t0 += step) {
    float rows[U][NV][4];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * RPW + r;
      load_row<VEC, LPR, NV>(logits + (t < T ? t : T - 1) * E, sub, E, -INFINITY, rows[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = t0 + u * RPW + r;
      const bool ok = t < T;
      const int64_t tt = ok ? t : T - 1;
      float(&l)[NV][4] = rows[u];
      const float ls = __ldg(lse + tt);
      const bool empty = ls == -INFINITY;
      const float ls0 = empty ? 0.f : ls;
      float g = 0.f;
      bool twice = false;
      if (dw != nullptr) {
        for (int j = sub; j < k; j += LPR) {
          const int id = __ldg(ids + tt * k + j);
          const bool in = id >= 0 && id < E;
          if (in) s_row[id] = __int_as_float(j);
          else if (ok) atomicCAS(status, 0, kErrBadIds);
          g = fmaf(__ldg(w + tt * k + j), __ldg(dw + tt * k + j), g);
        }
        g = lanes_sum<LPR>(g);
        __syncwarp();
        for (int j = sub; j < k; j += LPR) {
          const int id = __ldg(ids + tt * k + j);
          if (id >= 0 && id < E) twice |= __float_as_int(s_row[id]) != j;
        }
        twice = __any_sync(0xffffffffu, twice);  // also: every read before the rows are written
      }
      float dot = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[i][e] = __expf(l[i][e] - ls0);
          sum += l[i][e];
          dot = fmaf(f[i][e], l[i][e], dot);
        }
      lanes_sums<LPR>(dot, sum);
      // P = exp(l - lse) over its own sum: the rounding of lse, |lse| 2^-24 of every P,
      // is common to the row and drops out
      const float inv = empty ? 0.f : __fdividef(1.f, sum);
      const float base = inv * fmaf(c_z, ls0, -c_aux * (dot * inv)), ca = c_aux * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l[i][e] *= fmaf(ca, f[i][e], base);
          if (!VEC && dw != nullptr) s_row[ecol<VEC, LPR>(sub, i, e)] = l[i][e];
        }
        if (VEC && dw != nullptr)
          *(reinterpret_cast<float4*>(s_row) + sub + LPR * i) =
              make_float4(l[i][0], l[i][1], l[i][2], l[i][3]);
      }
      if (dw != nullptr) {
        __syncwarp();
        for (int q = 0; q < (twice ? LPR : 1); ++q) {  // one lane of a row after the other, or all
          if (!empty && (!twice || sub == q))
            for (int j = sub; j < k; j += LPR) {
              const int id = __ldg(ids + tt * k + j);
              if (id >= 0 && id < E)
                s_row[id] += __ldg(w + tt * k + j) * (__ldg(dw + tt * k + j) - g);
            }
          __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (VEC) {
            const float4 v = *(reinterpret_cast<const float4*>(s_row) + sub + LPR * i);
            l[i][0] = v.x; l[i][1] = v.y; l[i][2] = v.z; l[i][3] = v.w;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) l[i][e] = s_row[ecol<VEC, LPR>(sub, i, e)];
          }
        }
        __syncwarp();  // read before the next turn writes its slot numbers
      }
      if (ok) {
        float* row = dlogits + t * E;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (VEC) {
            if (ecol<VEC, LPR>(sub, i, 0) < E)
              *(reinterpret_cast<float4*>(row) + sub + LPR * i) =
                  make_float4(l[i][0], l[i][1], l[i][2], l[i][3]);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int c = ecol<VEC, LPR>(sub, i, e);
              if (c < E) row[c] = l[i][e];
            }
          }
        }
      }
    }
  }
}

struct RouterLaunch {
  const float* logits;
  int T, E, k;
  const int32_t *counts, *ids;
  const float *w, *dw;
  float* lse;
  float *losses, *pmean, *part, *dlogits;
  float aux_coef, z_coef;
  int* status;
  bool bwd;
  cudaStream_t s;
};

// Vectors of 4 logits a row is held in: a power of two.
int row_vectors(int E) {
  int v = 1;
  while (4 * v < E) v *= 2;
  return v;
}
// 16 logits a lane, and no lane with two rows that it holds alone.
int rows_per_warp(int E) { return std::min(32, std::max(1, 128 / row_vectors(E))); }
int row_blocks(int T, int E) {
  const int per = kRouterWarps * rows_per_warp(E);
  return static_cast<int>(std::min<int64_t>((static_cast<int64_t>(T) + per - 1) / per, kRouterBlocks));
}
int part_ld(int E) { return (E + 1 + 3) / 4 * 4; }
bool one_launch(int T, int E) { return E <= kOneMaxE && static_cast<int64_t>(T) * E <= kOneMaxLogits; }

template <bool VEC, int LPR, int NV>
cudaError_t loss(const RouterLaunch& q) {
  const int ld = part_ld(q.E);
  const LossEnd end{q.counts, q.k, q.losses, q.pmean};
  if constexpr (LPR * NV <= kOneMaxE / 4) {
    if (one_launch(q.T, q.E)) {
      const int64_t per = kOneThreads / 32 * rows_per_warp(q.E);
      const int64_t need = (static_cast<int64_t>(q.T) + per - 1) / per;
      unsigned blocks = 1;
      while (blocks < kOneBlocks && blocks < need) blocks *= 2;
      return launch_pdl_cluster(router_loss_kernel<VEC, LPR, NV, true>, dim3(blocks),
                                dim3(kOneThreads), static_cast<size_t>(kOneThreads / 32) * ld * 4, q.s,
                                blocks, q.logits, q.T, q.E, q.lse, q.part, ld, end);
    }
  }
  const int blocks = row_blocks(q.T, q.E);
  const cudaError_t e = launch_pdl(router_loss_kernel<VEC, LPR, NV, false>, dim3(blocks),
                                   dim3(kRouterThreads), static_cast<size_t>(kRouterWarps) * ld * 4,
                                   q.s, q.logits, q.T, q.E, q.lse, q.part, ld, end);
  if (e != cudaSuccess) return e;
  return launch_pdl_cluster(router_loss_final_kernel, dim3(kFinalBlocks), dim3(kFinalThreads), 0, q.s,
                            kFinalBlocks, static_cast<const float*>(q.part), blocks, ld, q.T, q.E, end);
}

template <bool VEC, int LPR, int NV>
cudaError_t grad(const RouterLaunch& q) {
  const float T = static_cast<float>(q.T);
  const size_t smem = q.dw != nullptr ? static_cast<size_t>(kRouterWarps) * 128 * NV * 4 : 0;
  return launch_pdl(router_bwd_kernel<VEC, LPR, NV>, dim3(row_blocks(q.T, q.E)), dim3(kRouterThreads),
                    smem, q.s, q.logits, static_cast<const float*>(q.lse), q.counts, q.ids, q.w, q.dw,
                    q.T, q.E, q.k, q.aux_coef * static_cast<float>(q.E) / T, 2.f * q.z_coef / T,
                    1.f / (T * static_cast<float>(q.k)), q.dlogits, q.status);
}

// Lanes and vectors of a row.  As few lanes as hold it with 4 vectors each: few
// lanes mean few shuffles for a sum.  But rows read by single logits (E no multiple
// of 4, or logits off a 16-byte boundary) take 8 lanes, and more of them at once, so
// that a load covers 32 bytes of a row: from 33 experts on for the losses, from 17
// for the gradient, which also writes so.  300,000 rows of 61, losses: 23.9 us
// against 27.5, gradient 46 against 62; 944,811 rows of 19: 41.2 against 33.2,
// gradient 91 against 136; 900,000 rows of 5, gradient: 79 against 17.
// 300,000 rows of 64, by vectors, with 8 lanes: 21.8 against 19.9.
template <bool VEC>
cudaError_t launch_loss(const RouterLaunch& q) {
  switch (row_vectors(q.E)) {
    case 1: return loss<VEC, 1, 1>(q);
    case 2: return loss<VEC, 1, 2>(q);
    case 4: return loss<VEC, 1, 4>(q);
    case 8: return loss<VEC, 2, 4>(q);
    case 16: return loss<VEC, VEC ? 4 : 8, VEC ? 4 : 2>(q);
    case 32: return loss<VEC, 8, 4>(q);
    case 64: return loss<VEC, 16, 4>(q);
    case 128: return loss<VEC, 32, 4>(q);
    default: return loss<VEC, 32, 8>(q);
  }
}
template <bool VEC>
cudaError_t launch_grad(const RouterLaunch& q) {
  switch (row_vectors(q.E)) {
    case 1: return grad<VEC, 1, 1>(q);
    case 2: return grad<VEC, 1, 2>(q);
    case 4: return grad<VEC, 1, 4>(q);
    case 8: return grad<VEC, VEC ? 2 : 8, VEC ? 4 : 1>(q);
    case 16: return grad<VEC, VEC ? 4 : 8, VEC ? 4 : 2>(q);
    case 32: return grad<VEC, 8, 4>(q);
    case 64: return grad<VEC, 16, 4>(q);
    case 128: return grad<VEC, 32, 4>(q);
    default: return grad<VEC, 32, 8>(q);
  }
}
cudaError_t launch_router(const RouterLaunch& q, bool vec) {
  if (q.bwd) return vec ? launch_grad<true>(q) : launch_grad<false>(q);
  return vec ? launch_loss<true>(q) : launch_loss<false>(q);
}

int bad(const char* msg) { return record_error(MOE_ERR_INVALID_ARG, msg); }
bool misaligned(const void* p, unsigned size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) != 0; }

int check_sizes(int32_t T, int32_t E, int32_t k) {
  if (T < 0 || E <= 0 || k <= 0 || k > E) return bad("bad T/E/k");
  if (E > kMaxExperts || k > 32) return record_error(MOE_ERR_UNSUPPORTED, "E > 1024 or k > 32");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_router_loss_workspace_size(int32_t T, int32_t E) {
  if (T < 0 || E <= 0 || E > kMaxExperts) return 0;
  return static_cast<size_t>(row_blocks(T, E)) * static_cast<size_t>(part_ld(E)) * 4;
}

int moe_router_loss_fwd(const float* logits, int32_t T, int32_t E, int32_t k, const int32_t* counts,
                        float* losses, float* lse, float* pmean, void* ws, size_t ws_bytes,
                        moe_stream_t stream) {
  NvtxScope nvtx("moe_router_loss_fwd");
  int rc = check_sizes(T, E, k);
  if (rc) return rc;
  if (T == 0) return bad("the mean over no tokens: T must be positive");
  if (!logits || !counts || !losses || !lse || !pmean || !ws) return bad("NULL pointer");
  if (misaligned(logits, 4) || misaligned(counts, 4) || misaligned(losses, 4) || misaligned(lse, 4) ||
      misaligned(pmean, 4) || misaligned(ws, 16))
    return bad("misaligned pointer");
  if (ws_bytes < moe_router_loss_workspace_size(T, E))
    return record_error(MOE_ERR_WORKSPACE, "router loss workspace too small");
  RouterLaunch q = {};
  q.logits = logits; q.T = T; q.E = E; q.k = k; q.lse = lse; q.part = static_cast<float*>(ws);
  q.counts = counts; q.losses = losses; q.pmean = pmean; q.s = stream;
  ProbeScope probe("router_loss", stream);
  const cudaError_t e = launch_router(q, E % 4 == 0 && !misaligned(logits, 16));
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

int moe_router_bwd(const float* logits, const float* lse, int32_t T, int32_t E, int32_t k,
                   const int32_t* counts, const int32_t* ids, const float* weights,
                   const float* dweights, float aux_coef, float z_coef, float* dlogits,
                   moe_stream_t stream) {
  NvtxScope nvtx("moe_router_bwd");
  int rc = check_sizes(T, E, k);
  if (rc) return rc;
  if (T == 0) return record_error(MOE_OK, "");
  if (!logits || !lse || !dlogits) return bad("NULL pointer");
  if (dweights != nullptr && (!ids || !weights)) return bad("dweights needs ids and weights");
  if (aux_coef != 0.f && !counts) return bad("the load-balancing loss needs counts");
  if (misaligned(logits, 4) || misaligned(lse, 4) || misaligned(dlogits, 4) || misaligned(counts, 4) ||
      misaligned(ids, 4) || misaligned(weights, 4) || misaligned(dweights, 4))
    return bad("misaligned pointer");
  RouterLaunch q = {};
  rc = device_status_word(&q.status);
  if (rc != MOE_OK) return rc;
  q.logits = logits; q.T = T; q.E = E; q.k = k; q.counts = counts; q.ids = ids; q.w = weights;
  q.dw = dweights; q.lse = const_cast<float*>(lse); q.dlogits = dlogits; q.aux_coef = aux_coef;
  q.z_coef = z_coef; q.bwd = true; q.s = stream;
  ProbeScope probe("router_bwd", stream);
  const cudaError_t e =
      launch_router(q, E % 4 == 0 && !misaligned(logits, 16) && !misaligned(dlogits, 16));
  if (e != cudaSuccess) return record_error(MOE_ERR_CUDA, cudaGetErrorString(e));
  return record_error(MOE_OK, "");
}

}  // extern "C"
