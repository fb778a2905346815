// Backward of norm_fwd.cu, in one pass over the rows.  With rh = r rstd_r,
// yh = y rstd_y, u = w_pre + off, q = w_post + off:
//   e = dr + rstd_r dn u,  c1 = mean(dn u rh),  t = e - rstd_r c1 rh        dx = t
//   p = yh q (or y);  dp = s a t;  dy = rstd_y (dp q - yh mean(dp p))      (or dp)
//   dgate = s a' t p, summed over what the gate is broadcast over
//   dw_pre = sum_rows dn rh;  dw_post = sum_rows dp yh
// t is linear in c1, so one reduction gives every row sum:
//   S1 = sum dn u rh,  S2 = sum A p e,  S3 = sum A p rh,
//   sum A p t = S2 - rstd_r c1 S3     (A = a(gate) where it varies along the row, else 1)
// Column sums are kept in registers over the rows of a block, written once as
// partials and added by a second kernel in a fixed order (no atomics).  Two
// give all three gradients: sum dn rh = dw_pre, and with Y = yh (or y)
//   no gate, token, element: S = sum a t Y,  dw_post = s S
//   channel:                 S = sum t Y,    dw_post = s a S,  dgate = s a' q S
// A row costs some 40 instructions for 8 columns and two waits for its sums, so
// rows overlap: several blocks on an SM, and a ring that loads ahead.  Bound by
// memory where the weights are frozen (32768x2880, fp32 stream, element gate:
// 328 us with 6.2 TB/s); with column sums by what an SM issues between a row's two
// barriers: channel gate, 4096x2048 29 us, 16384x2048 83 us, 4.3 ns a further row
// (0.84 of a plain copy's rate; with frozen weights 4.0).  Of the 29 us the second
// kernel takes 4, and loading the factors, filling the ring and writing the partial
// sums about 7.  Rows read directly, above 8192 columns: 0.4 to 0.5, latency and
// registers (4096x12000 in bf16: 371 us).
#pragma once

#include "norm.cuh"

namespace moe {

// The two families, compiled apart: rows read directly (any width, alignment
// and gate; column sums always kept) and rows through the ring.
cudaError_t launch_norm_bwd_direct(const NormArgs& a, int x_type, int y_type, bool vec, int blocks,
                                   cudaStream_t s);
cudaError_t launch_norm_bwd_ring(const NormArgs& a, int x_type, int y_type, bool vec, int blocks,
                                 cudaStream_t s);

// MAXT, MINB: threads of a block at most, blocks an SM holds at least.
template <typename XT, typename YT, bool VEC, int NV, int GATE, bool SUMS, bool RING, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_bwd_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t s_tiles[];
  __shared__ float s_red[2][16][4];
  __shared__ RingState s_ring;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.W, groups = (blockDim.x >> 5) / W;
  const int grp = warp / W, first = grp * W;
  const int v0 = (warp - first) * 32 + lane;
  const int d = a.d;
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const bool channel = gate_is<GATE>(a.gate_kind, MOE_GATE_CHANNEL);
  const bool element = gate_is<GATE>(a.gate_kind, MOE_GATE_ELEMENT);
  const bool sum_gate_row = a.gate_kind == MOE_GATE_TOKEN && a.dgate != nullptr;
  const float inv_d = 1.f / static_cast<float>(d);
  const RingSrc src[kRingSrcs] = {{a.x, sizeof(XT)},
                                  {pre ? a.r : nullptr, sizeof(XT)},
                                  {pre ? a.n : nullptr, sizeof(YT)},
                                  {a.y, sizeof(YT)},
                                  {element ? a.gate : nullptr, sizeof(YT)}};
  bool ahead = false;
  if (!RING && NV >= 2) {
    int size = 0;
    for (int i = 0; i < kRingSrcs; ++i) size += src[i].p != nullptr ? src[i].esize : 0;
    ahead = size * d <= kPrefetchBytes;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
  f2 acc_y[NV][4], acc_r[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc_y[i][e] = acc_r[i][e] = pk(0.f);
  if (RING) {
    if (threadIdx.x == 0) ring_init(s_ring, a.stages);
    __syncthreads();
  }
  pdl_wait();
  if (RING && threadIdx.x == 0)
    for (int q = 0; q < a.stages && base + q * step < a.T; ++q)
      ring_fill<VEC>(src, s_tiles + q * a.tile, &s_ring.full[q], base + q * step, a.T, groups, d);
  // per column: k = (w_post + off) a(channel gate), u = w_pre + off
  auto make_k = [&](int v, f2 (&k)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) k[e] = pk(1.f);
    if (post) {
      get8<float, VEC>(a.w_post, v, d, k);
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = add2(k[e], pk(a.w_off));
    }
    if (channel) {
      f2 g[4];
      get8<float, VEC>(static_cast<const float*>(a.gate), v, d, g);
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = mul2(k[e], gate_pair(g[e], a.sigmoid));
    }
  };
  auto make_u = [&](int v, f2 (&u)[4]) {
    get8<float, VEC>(a.w_pre, v, d, u);
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = add2(u[e], pk(a.w_off));
  };
  // Kept for all rows: in shared memory behind the ring (registers are what
  // limits the blocks on an SM), in registers without one, or made again.
  constexpr bool kKeep = !RING && NV == 1;
  f2 ck[kKeep ? 4 : 1], cu[kKeep ? 4 : 1];
  float4* s_const = reinterpret_cast<float4*>(s_tiles + a.stages * a.tile) + threadIdx.x;
  const int nthr = blockDim.x;
  if (RING || kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      f2 k[4], u[4];
      if (has_y) make_k(v0 + i * 32 * W, k);
      if (pre) make_u(v0 + i * 32 * W, u);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (!has_y) k[e] = pk(0.f);
        if (!pre) u[e] = pk(0.f);
        if (kKeep) ck[kKeep ? e : 0] = k[e], cu[kKeep ? e : 0] = u[e];
      }
      if (RING) {
        Raw8<float> q;
        narrow(k, q);
        s_const[(4 * i) * nthr] = q.a;
        s_const[(4 * i + 1) * nthr] = q.b;
        narrow(u, q);
        s_const[(4 * i + 2) * nthr] = q.a;
        s_const[(4 * i + 3) * nthr] = q.b;
      }
    }
  }
  auto get_const = [&](int i, int which, f2 (&f)[4]) {  // which: 0 k, 1 u
    if (RING) {
      Raw8<float> q;
      q.a = s_const[(4 * i + 2 * which) * nthr];
      q.b = s_const[(4 * i + 2 * which + 1) * nthr];
      widen(q, f);
    } else if (kKeep) {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = which ? cu[kKeep ? e : 0] : ck[kKeep ? e : 0];
    } else if (which) {
      make_u(v0 + i * 32 * W, f);
    } else {
      make_k(v0 + i * 32 * W, f);
    }
  };
  // offsets of each input's rows in a tile
  const int place_x = ring_place<VEC>(groups * d * static_cast<int>(sizeof(XT))),
            place_y = ring_place<VEC>(groups * d * static_cast<int>(sizeof(YT)));
  const int at_r = a.x != nullptr ? place_x : 0, at_n = at_r + (pre ? place_x : 0),
            at_y = at_n + (pre ? place_y : 0), at_g = at_y + (has_y ? place_y : 0);
  // the scalars of a row are read one tile ahead
  float next_r = 0.f, next_y = 0.f, next_g = 0.f;
  auto read_ahead = [&](int64_t row) {
    const bool in = row < a.T;
    next_r = pre && in ? a.rstd_r[row] : 0.f;
    next_y = !post ? 1.f : in ? a.rstd_y[row] : 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN) next_g = in ? static_cast<const float*>(a.gate)[row] : 0.f;
  };
  read_ahead(base + grp);
  int turn = 0, stage = 0, phase = 0, before = 0;
  bool filling = true;
  for (; base < a.T; base += step, turn ^= 1) {
    const int64_t row = base + grp;
    const bool ok = row < a.T;
    const int64_t off = ok ? row * d : 0;
    const int dd = ok ? d : 0;
    if (ahead && v0 == 0 && row + step < a.T) prefetch_row(src, row + step, d);
    const XT* pdr = static_cast<const XT*>(a.x) + off;
    const XT* pr = static_cast<const XT*>(a.r) + off;
    const YT* pdn = static_cast<const YT*>(a.n) + off;
    const YT* py = static_cast<const YT*>(a.y) + off;
    const YT* pg = static_cast<const YT*>(a.gate) + off;
    const float rs_r = next_r, rs_y = next_y;
    float a_row = 1.f, da_row = 0.f;
    if (a.gate_kind == MOE_GATE_TOKEN) gate_value(next_g, a.sigmoid, a_row, da_row);
    read_ahead(row + step);
    if constexpr (RING) {
      if (!ring_wait(s_ring, &s_ring.full[stage], stage, phase, base, a.status, kWaitTimeoutNs)) filling = false;
      const uint8_t* t = s_tiles + stage * a.tile;
      pdr = ring_row<VEC>(t, static_cast<const XT*>(a.x), base, d) + grp * d;
      pr = ring_row<VEC>(t + at_r, static_cast<const XT*>(a.r), base, d) + grp * d;
      pdn = ring_row<VEC>(t + at_n, static_cast<const YT*>(a.n), base, d) + grp * d;
      py = ring_row<VEC>(t + at_y, static_cast<const YT*>(a.y), base, d) + grp * d;
      pg = ring_row<VEC>(t + at_g, static_cast<const YT*>(a.gate), base, d) + grp * d;
    }
    // pass 1: e in place of dr; the row sums, of r and y as they are (their rstd
    // factors follow)
    constexpr bool kAgain = NV >= 2;  // pass 2 reads r and y again: registers
    constexpr int NK = kAgain ? 1 : NV;
    f2 ev[NV][4], r_[NK][4], y_[NK][4];
    f2 sum_g = pk(0.f), sum_e = pk(0.f), sum_h = pk(0.f);
    const f2 rs_r2 = pk(rs_r);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      if (col_of<VEC>(v, 0) >= dd) continue;  // no column of this share
      f2 k[4], dn[4];
      f2(&r)[4] = r_[kAgain ? 0 : i];
      f2(&y)[4] = y_[kAgain ? 0 : i];
      if (a.x != nullptr) {
        get8<XT, VEC>(pdr, v, d, ev[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) ev[i][e] = pk(0.f);
      }
      if (has_y) get8<YT, VEC>(py, v, d, y);
      if (pre) {
        get8<XT, VEC>(pr, v, d, r);
        get8<YT, VEC>(pdn, v, d, dn);
        get_const(i, 1, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (SUMS) acc_r[i][e] = fma2(dn[e], mul2(r[e], rs_r2), acc_r[i][e]);
          const f2 g = mul2(dn[e], k[e]);
          ev[i][e] = fma2(rs_r2, g, ev[i][e]);
          sum_g = fma2(g, r[e], sum_g);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = pk(0.f);
      }
      if (post || sum_gate_row) {
        get_const(i, 0, k);
        if (element) get8<YT, VEC>(pg, v, d, dn);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f2 ap = mul2(y[e], k[e]);
          if (element) ap = mul2(ap, gate_pair(dn[e], a.sigmoid));
          sum_e = fma2(ap, ev[i][e], sum_e);
          sum_h = fma2(ap, r[e], sum_h);
        }
      }
    }
    float sum[3] = {sum2(sum_g), sum2(sum_e), sum2(sum_h)};
    if (pre || post || sum_gate_row) row_sum<3>(sum, s_red[turn], W, warp, first);
    if (RING && threadIdx.x == 0 && filling && base >= step) {  // the previous tile's place is free
      const int64_t next = base + (a.stages - 1) * step;
      if (next < a.T) ring_fill<VEC>(src, s_tiles + before * a.tile, &s_ring.full[before], next, a.T, groups, d);
    }
    const float c1 = rs_r * (rs_r * (rs_r * (sum[0] * inv_d)));  // t = e - c1 r
    const float apt = rs_y * fmaf(-c1, sum[2], sum[1]);     // sum A p t
    if (sum_gate_row && ok && v0 == 0)
      static_cast<float*>(a.dgate)[row] = a.scale * da_row * apt;
    const float fac = a.scale * a_row;                      // dp = fac A t
    const float c2 = post ? fac * apt * inv_d * rs_y * rs_y : 0.f;  // dy = rstd_y fac k t - c2 y
    const f2 c1n = pk(-c1), c2n = pk(-c2), facy = pk(fac * rs_y), ry2 = pk(a_row * rs_y);
    // pass 2: the outputs
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      if (col_of<VEC>(v, 0) >= dd) continue;
      f2 k[4], o[4];
      f2(&r)[4] = r_[kAgain ? 0 : i];
      f2(&y)[4] = y_[kAgain ? 0 : i];
      if (kAgain) {
        if (pre) get8<XT, VEC>(pr, v, d, r);
        if (has_y) get8<YT, VEC>(py, v, d, y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) ev[i][e] = fma2(c1n, r[e], ev[i][e]);  // t
      if (a.dx != nullptr) put8<XT, VEC>(static_cast<XT*>(a.dx) + off, v, d, ev[i]);
      if (!has_y) continue;
      get_const(i, 0, k);
      f2 g[4], dg[4];
      if (element) {
        get8<YT, VEC>(pg, v, d, g);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 gv = unpk(g[e]);
          float a0, a1, d0, d1;
          gate_value(gv.x, a.sigmoid, a0, d0);
          gate_value(gv.y, a.sigmoid, a1, d1);
          g[e] = pk(a0, a1);
          dg[e] = pk(d0, d1);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f2 at = element ? mul2(g[e], ev[i][e]) : ev[i][e];
        const f2 yh = mul2(y[e], ry2);  // a_row Y
        if (SUMS) acc_y[i][e] = fma2(at, yh, acc_y[i][e]);
        o[e] = mul2(mul2(at, k[e]), facy);
        if (post) o[e] = fma2(y[e], c2n, o[e]);
        if (element) dg[e] = mul2(mul2(dg[e], mul2(ev[i][e], pk(a.scale))), mul2(yh, k[e]));
      }
      if (a.dy != nullptr) put8<YT, VEC>(static_cast<YT*>(a.dy) + off, v, d, o);
      if (element && a.dgate != nullptr) put8<YT, VEC>(static_cast<YT*>(a.dgate) + off, v, d, dg);
    }
    before = stage;
    if (++stage == a.stages) { stage = 0; phase ^= 1; }
  }
  if (RING) ring_drain(s_ring, a.stages, step, a.T);
  if (!SUMS) return;
  float* part = a.part + (static_cast<int64_t>(blockIdx.x) * groups + grp) * a.nsum * d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = v0 + i * 32 * W;
    if (a.sum_y >= 0) put8<float, VEC>(part + static_cast<int64_t>(a.sum_y) * d, v, d, acc_y[i]);
    if (a.sum_r >= 0) put8<float, VEC>(part + static_cast<int64_t>(a.sum_r) * d, v, d, acc_r[i]);
  }
}

}  // namespace moe
