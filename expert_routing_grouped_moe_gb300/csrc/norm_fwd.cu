// Norm after a block, gated and scaled residual sum, norm before the next
// block, in one pass over the rows:
//   p = y rstd(y) (w_post + off) or y;  r = x + s a(gate) p;  n = r rstd(r) (w_pre + off)
// with rstd(z) = 1/sqrt(mean z^2 + eps).  Everything between the loads and the
// stores is fp32; n is the norm of the unrounded r.
// Bound by memory: x and y are read once, r and n written once, a row waits in
// registers for its two sums.  16384x2048 in bf16: 42 us, 6.4 TB/s (0.94 of a plain
// copy's rate); 4096x2048: 12.5 us, 0.79 (27 rows an SM: filling the ring and the
// last rows are 3 us of it); one row of 2048: 2.4 us, a launch.
#include "norm.cuh"

namespace moe {
namespace {

// RING: rows come through the ring of bulk copies (at least one norm, rows of
// several warps); else each thread loads its share from memory.
template <typename XT, typename YT, bool VEC, int NV, int GATE, bool RING>
__global__ void __launch_bounds__(RING && NV == 1 ? 384 : 512, RING && NV == 1 ? 2 : 1) norm_fwd_kernel(const NormArgs a) {
  extern __shared__ __align__(128) uint8_t s_tiles[];
  __shared__ float s_red[2][16][4];
  __shared__ RingState s_ring;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.W, groups = (blockDim.x >> 5) / W;
  const int grp = warp / W, first = grp * W;
  const int v0 = (warp - first) * 32 + lane;  // share numbers v0 + i * 32 W
  const int d = a.d;
  const bool has_y = a.y != nullptr, post = a.w_post != nullptr, pre = a.w_pre != nullptr;
  const float inv_d = 1.f / static_cast<float>(d);
  const RingSrc src[kRingSrcs] = {
      {a.x, sizeof(XT)}, {a.y, sizeof(YT)},
      {gate_is<GATE>(a.gate_kind, MOE_GATE_ELEMENT) ? a.gate : nullptr, sizeof(YT)}, {nullptr, 0},
      {nullptr, 0}};
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  int64_t base = static_cast<int64_t>(blockIdx.x) * groups;
  if (RING) {
    if (threadIdx.x == 0) ring_init(s_ring, a.stages);
    __syncthreads();
  }
  pdl_wait();
  if (RING && threadIdx.x == 0)
    for (int q = 0; q < a.stages && base + q * step < a.T; ++q)
      ring_fill<VEC>(src, s_tiles + q * a.tile, &s_ring.full[q], base + q * step, a.T, groups, d);
  const bool channel = gate_is<GATE>(a.gate_kind, MOE_GATE_CHANNEL);
  const bool element = gate_is<GATE>(a.gate_kind, MOE_GATE_ELEMENT);
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
  RowConst<NV> ck, cu;
  if (NV <= 2) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (has_y) make_k(v0 + i * 32 * W, ck.f[NV <= 2 ? i : 0]);
      if (pre) make_u(v0 + i * 32 * W, cu.f[NV <= 2 ? i : 0]);
    }
  }
  // a token's gate is read one tile ahead
  const float* tokens = a.gate_kind == MOE_GATE_TOKEN ? static_cast<const float*>(a.gate) : nullptr;
  float next_g = tokens && base + grp < a.T ? tokens[base + grp] : 0.f;
  int turn = 0;  // which of the two arrays the next row sum uses
  int stage = 0, phase = 0, before = 0;
  bool filling = true;
  for (; base < a.T; base += step) {
    const int64_t row = base + grp;
    const bool ok = row < a.T;
    const int64_t off = ok ? row * d : 0;
    const int dd = ok ? d : 0;  // no column of a row past the end
    const XT* px = static_cast<const XT*>(a.x) + off;
    const YT* py = static_cast<const YT*>(a.y) + off;
    const YT* pg = static_cast<const YT*>(a.gate) + off;
    if constexpr (RING) {
      if (!ring_wait(s_ring, &s_ring.full[stage], stage, phase, base, a.status, kWaitTimeoutNs)) filling = false;
      const uint8_t* t = s_tiles + stage * a.tile;
      px = ring_row<VEC>(t, static_cast<const XT*>(a.x), base, d) + grp * d;
      if (a.x != nullptr) t += ring_place<VEC>(groups * d * sizeof(XT));
      py = ring_row<VEC>(t, static_cast<const YT*>(a.y), base, d) + grp * d;
      if (has_y) t += ring_place<VEC>(groups * d * sizeof(YT));
      pg = ring_row<VEC>(t, static_cast<const YT*>(a.gate), base, d) + grp * d;
    }
    // after the first barrier of this tile: the previous tile's place is free
    auto refill = [&]() {
      if (RING && threadIdx.x == 0 && filling && base >= step) {
        const int64_t next = base + (a.stages - 1) * step;
        if (next < a.T) ring_fill<VEC>(src, s_tiles + before * a.tile, &s_ring.full[before], next, a.T, groups, d);
      }
    };
    f2 x[NV][4], y[NV][4];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = v0 + i * 32 * W;
      get8<XT, VEC>(px, v, a.x != nullptr ? dd : 0, x[i]);
      get8<YT, VEC>(py, v, has_y ? dd : 0, y[i]);
    }
    if (has_y) {
      float rs = 1.f;
      if (post) {
        f2 ss = pk(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = fma2(y[i][e], y[i][e], ss);
        float sum[1] = {sum2(ss)};
        row_sum<1>(sum, s_red[turn], W, warp, first);
        turn ^= 1;
        refill();
        rs = rsqrtf(fmaf(sum[0], inv_d, a.eps));
        if (ok && v0 == 0) a.rstd_y[row] = rs;
      }
      float fac = a.scale * rs;
      if (tokens) {
        float g, dg;
        gate_value(next_g, a.sigmoid, g, dg);
        fac *= g;
        next_g = row + step < a.T ? tokens[row + step] : 0.f;
      }
      const f2 fac2 = pk(fac);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * 32 * W;
        f2 k[4];
        if (NV > 2) make_k(v, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], NV > 2 ? k[e] : ck.f[NV <= 2 ? i : 0][e]);
        if (element) {
          get8<YT, VEC>(pg, v, dd, k);
#pragma unroll
          for (int e = 0; e < 4; ++e) y[i][e] = mul2(y[i][e], gate_pair(k[e], a.sigmoid));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) x[i][e] = fma2(fac2, y[i][e], x[i][e]);
        put8<XT, VEC>(static_cast<XT*>(a.r) + off, v, dd, x[i]);
      }
    }
    if (pre) {
      f2 ss = pk(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) ss = fma2(x[i][e], x[i][e], ss);
      float sum[1] = {sum2(ss)};
      row_sum<1>(sum, s_red[turn], W, warp, first);
      turn ^= 1;
      if (!post) refill();
      const float rs = rsqrtf(fmaf(sum[0], inv_d, a.eps));
      if (ok && v0 == 0) a.rstd_r[row] = rs;
      const f2 rs2 = pk(rs);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = v0 + i * 32 * W;
        f2 u[4];
        if (NV > 2) make_u(v, u);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[i][e] = mul2(mul2(x[i][e], rs2), NV > 2 ? u[e] : cu.f[NV <= 2 ? i : 0][e]);
        put8<YT, VEC>(static_cast<YT*>(a.n) + off, v, dd, x[i]);
      }
    }
    before = stage;
    if (++stage == a.stages) { stage = 0; phase ^= 1; }
  }
  if (RING) ring_drain(s_ring, a.stages, step, a.T);
}

template <typename XT, typename YT, bool VEC, int NV, int GATE, bool RING>
cudaError_t go(const NormArgs& args, cudaStream_t s) {
  NormArgs a = args;
  const NormShape sh = norm_fwd_shape(a.d);
  auto kern = norm_fwd_kernel<XT, YT, VEC, NV, GATE, RING>;
  if (RING) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_ring(kern, done);
    if (e != cudaSuccess) return e;
  }
  // blocks whose registers fit an SM, found once for each block size
  static std::atomic<int> fit[kNormMaxWarps + 1];
  int per = fit[sh.threads() / 32].load(std::memory_order_relaxed);
  if (per == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kern, sh.threads(), 0);
    if (e != cudaSuccess) return e;
    if (per < 1) per = 1;
    fit[sh.threads() / 32].store(per, std::memory_order_relaxed);
  }
  if (RING) a.stages = ring_stages(a.tile, &per, 0, kFwdFlight);
  const int64_t need = (a.T + sh.groups - 1) / sh.groups;
  const int64_t most = static_cast<int64_t>(per) * kSMs;
  return launch_pdl(kern, dim3(static_cast<unsigned>(need < most ? need : most)), dim3(sh.threads()),
                    static_cast<size_t>(a.stages) * a.tile, s, a);
}

template <typename XT, typename YT, int NV>
cudaError_t pick_nv(const NormArgs& a, bool vec, cudaStream_t s) {
  if constexpr (NV <= 2)
    if (vec && a.tile > 0) switch (gate_class(a.gate_kind)) {
        case kGateRow: return go<XT, YT, true, NV, kGateRow, true>(a, s);
        case kGateChannel: return go<XT, YT, true, NV, kGateChannel, true>(a, s);
        default: return go<XT, YT, true, NV, kGateElement, true>(a, s);
      }
  if constexpr (NV <= 2)
    if (!vec && a.tile > 0) return go<XT, YT, false, NV, kGateAny, true>(a, s);
  return vec ? go<XT, YT, true, NV, kGateAny, false>(a, s)
             : go<XT, YT, false, NV, kGateAny, false>(a, s);
}

template <typename XT, typename YT>
cudaError_t pick(NormArgs a, bool vec, cudaStream_t s) {
  const NormShape sh = norm_fwd_shape(a.d);
  const int groups = sh.groups, nv = sh.nv;
  a.W = sh.W;
  auto place = [&](size_t size) {
    const int bytes = groups * a.d * static_cast<int>(size);
    return vec ? ring_place<true>(bytes) : ring_place<false>(bytes);
  };
  a.tile = (a.x ? place(sizeof(XT)) : 0) + (a.y ? place(sizeof(YT)) : 0) +
           (a.gate_kind == MOE_GATE_ELEMENT ? place(sizeof(YT)) : 0);
  const bool ring = nv <= 2 && a.W > 1 && (a.w_post || a.w_pre) &&
                    a.T > static_cast<int64_t>(kNormRingTiles) * groups;
  a.stages = 0;
  if (!ring || 2 * a.tile > kRingBytes) a.tile = 0;  // rows are read directly
  switch (nv) {
    case 1: return pick_nv<XT, YT, 1>(a, vec, s);
    case 2: return pick_nv<XT, YT, 2>(a, vec, s);
    default: return pick_nv<XT, YT, 4>(a, vec, s);
  }
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs& a, int x_type, int y_type, bool vec, cudaStream_t s) {
  if (a.T == 0) return cudaSuccess;
  if (x_type == MOE_BF16) return pick<bf16_t, bf16_t>(a, vec, s);
  return y_type == MOE_BF16 ? pick<float, bf16_t>(a, vec, s) : pick<float, float>(a, vec, s);
}

}  // namespace moe
