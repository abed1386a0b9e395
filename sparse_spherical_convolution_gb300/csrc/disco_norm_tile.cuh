// disco_norm_tile.cuh -- the channel norm by tiles (disco_norm.cuh): one pass
// over the data.  Instantiated without the 8-bit copy in disco_norm_tile.cu, with
// it in disco_norm_q.cu and disco_norm_q_any.cu.
//
// Bound by HBM: x and residual read once, h, y, q and scales written once.  A
// thread's V x NCH sums x + residual stay in fp32 registers between the
// statistics and the outputs, so y and q are computed from the unrounded h, while
// its shared memory already takes in the next tile (cp.async).  Without that
// prefetch, at the same occupancy, [2,128,361x720] took 114 us, with it 88.
//
// Measured (calls, GB300; the copy rate of this card is 6.78 TB/s):
//   [1,512,360x720] bf16, residual, h and y         174 us  6.1 TB/s, DRAM 75 % busy
//   [2,128,361x720] bf16, the same and q, groups 32 101 us  6.0 TB/s, DRAM 70 %
//   [14,54,20000] fp32, residual                     41 us  5.9 TB/s
//   [20,64,65343] bf16 (odd rows), residual         112 us  6.0 TB/s (111 for 65344)
//   [12,6,379015] fp32 (odd rows), residual         118 us  3.7 TB/s: channels come in
//     blocks of 16 (32 for 16 bits), 10 of a block's 16 places hold none of the 6
//   [3,80,181x361] fp16, no residual                 23 us  2.8 TB/s: it lies in L2,
//     and with 11 tiles to a CTA the latency of a tile's joins shows; one CTA of 384
//     threads to an SM (the planner's 512 threads, whatever a kernel's registers)
//   [2,128,361x719] bf16 (odd rows), residual and q 147 us  4.1 TB/s
// With q where a lane's channels or a CTA straddle groups, maxima are shared-memory
// atomics: [1,256,361x719] bf16, groups of 32, 244 us (2.5 TB/s); [3,433,11250],
// groups of 128, 49 us; fp32 [1,171,238050], groups of 55, 171 us.
// 512 channels of 518 KB rows take a pair of CTAs with 256-byte row pieces: 128-byte
// pieces in one CTA took 186 to 204 us (each piece lies in another 2 MB page).

#pragma once

#include "disco_norm.cuh"

namespace disco {
namespace norm {

// How the group maxima of the 8-bit copy are found: not at all; from one row
// of shared memory for each channel lane (a thread's channels and a group's
// CTAs are one); or by atomic maxima (any group size).
enum { kNoQ = 0, kRowsQ = 1, kAtomicQ = 2 };

template <typename T, int NCH, int Q, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads) norm_tile_kernel(const NormArgs a, const Tiling g, const int ng_max) {
  constexpr int V = 16 / (int)sizeof(T);
  using L = Lane<T, V, NCH, SHIFT>;
  using W = typename L::W;
  using Join = Joiner<V, 1, 1, SHIFT>;
  extern __shared__ __align__(16) char smem[];
  const uint32_t rank = g.CL > 1 ? cluster_rank() : 0;
  float* fsm = (float*)(smem + L::words(g) * 16 * 2);
  const Join J(g, fsm, rank);
  const int NT = g.NT, slots = J.slots, first_c = (int)rank * g.cpc;
  const L lane(g, a.B, a.C, a.P, J.lx, J.j, first_c, smem);
  const int nc = lane.nc;
  const T *x = (const T*)a.x, *res = (const T*)a.res, *w = (const T*)a.w;
  // Tiles fetched ahead: one of two tensors or two of one, about 64 KB in flight to
  // an SM either way ([4,128,361x720] without residual 86 us, one ahead 100).  Odd
  // rows are bound by instructions: one (22.6 us for [3,80,181x361], two 24.5).
  const int depth = res || SHIFT ? 1 : 2;
  W *rx = lane.slot, *rr = rx + L::words(g);

  float wt[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    wt[i] = i < nc && w ? to_f32(w[lane.channel(i)]) : 1.0f;
    if (i >= nc) {  // channels past the last: zeros, never copied over
      memset(rx + i * lane.stride, 0, 16);
      memset(rr + i * lane.stride, 0, 16);
    }
  }
  float* gmax = fsm + Join::floats(g);  // kRowsQ: [channel lane][slots]
  float* ginv = gmax + (Q == kRowsQ ? J.rows : 2 * ng_max) * slots;  // [group of this CTA][slots]
  uint32_t* gm = (uint32_t*)gmax;       // kAtomicQ: [2][group that touches this CTA][slots], the last tiles' in turn
  const int gm_half = ng_max * slots;
  int grp[NCH];  // kAtomicQ: the groups of this thread's channels
  if constexpr (Q == kAtomicQ) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) grp[i] = lane.channel(i) / a.G;
    for (int k = threadIdx.x; k < 2 * gm_half; k += NT) gm[k] = 0u;
  }

  Cursor at(g, a.C, a.P, blockIdx.x / g.CL), ahead = at;
  auto fetch = [&](W* to) {
    lane.fetch(g, ahead, x, to);
    if (res) lane.fetch(g, ahead, res, rr);
    copy_commit();
    ahead.next(g);
  };
  fetch(rx);
  if (depth == 2) fetch(rr);
  if (g.CL > 1) cluster_barrier();  // every CTA runs before another writes its shared memory

  for (int parity = 0; at.t < g.tiles; at.next(g), parity ^= 1) {
    const int n = (int)min((long long)g.TP, a.P - at.pos), m = lane.skew(at);  // n: pixels of the tile
    W* from = depth == 2 && parity ? rr : rx;
    F<V> v[NCH], s[1] = {fill<V>(0.0f)}, r[1];
    if (depth == 2) copy_wait<1>();
    else copy_wait<0>();
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      v[i] = unpack<T, V>(lane.read(from, i));
      if (res) v[i] = add(v[i], unpack<T, V>(lane.read(rr, i)));
    }
    fetch(from);
#pragma unroll
    for (int i = 0; i < NCH; ++i) s[0] = fma(v[i], v[i], s[0]);
    auto finish = [&](const float(&z)[1], float(&out)[1]) { out[0] = inverse_rms(z[0], a.inv_C, a.eps); };
    J.submit(s, m, parity, finish);
    if (a.h)
#pragma unroll
      for (int i = 0; i < NCH; ++i) lane.write(a.h, at, m, i, packed<T, V>(v[i]), n);
    J.collect(r, m, parity, finish);
#pragma unroll
    for (int i = 0; i < NCH; ++i) v[i] = mul(mul(v[i], r[0]), fill<V>(wt[i]));
    if (a.y)
#pragma unroll
      for (int i = 0; i < NCH; ++i) lane.write(a.y, at, m, i, packed<T, V>(v[i]), n);

    if constexpr (Q == kRowsQ) {
      F<V> top = fill<V>(0.0f);
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc)
#pragma unroll
          for (int e = 0; e < V; ++e) top.v[e] = fmaxf(top.v[e], fabsf(v[i].v[e]));  // a NaN does not count
      J.put(gmax + J.j * slots, top, m);
      __syncthreads();
      const int g0 = first_c / a.G, lanes = a.NG == 1 ? J.rows : a.G / NCH;
      for (int k = threadIdx.x; k < ng_max * n; k += NT) {
        const int gl = k / n, px = k - gl * n, to = J.slot(px);
        const int r0 = gl * lanes, r1 = min(r0 + lanes, J.rows);
        float t = kAmaxFloor;
        for (int z = r0; z < r1; ++z) t = fmaxf(t, gmax[z * slots + to]);
        ginv[gl * slots + to] = kE4m3Max / t;
        if (g0 + gl < a.NG) a.scale[(at.b * a.NG + g0 + gl) * a.P + at.pos + px] = t / kE4m3Max;
      }
      __syncthreads();
      const F<V> inv = J.get(ginv + min(J.j / lanes, ng_max - 1) * slots, m);
#pragma unroll
      for (int i = 0; i < NCH; ++i) lane.write(a.q, at, m, i, packed_e4m3<V>(mul(v[i], inv)), n);
    }

    if constexpr (Q == kAtomicQ) {
      const int last_c = min(first_c + g.cpc, a.C) - 1, g0 = first_c / a.G;
      const int ng = last_c >= first_c ? last_c / a.G - g0 + 1 : 0;
      uint32_t* mx = gm + parity * gm_half;
      F<V> top = fill<V>(0.0f);
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc) {
#pragma unroll
          for (int e = 0; e < V; ++e) top.v[e] = fmaxf(top.v[e], fabsf(v[i].v[e]));  // a NaN does not count
          if (i == nc - 1 || grp[i] != grp[i + 1 < NCH ? i + 1 : i]) {
            uint32_t* to = mx + (grp[i] - g0) * slots;
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (lane.in(e, m, n)) atomicMax(to + J.slot(J.lx * V - m + e), __float_as_uint(top.v[e]));
            top = fill<V>(0.0f);
          }
        }
      if (g.CL > 1) cluster_barrier();
      else __syncthreads();
      for (int k = threadIdx.x; k < ng * n; k += NT) {
        const int gl = k / n, px = k - gl * n, of = g0 + gl, to = J.slot(px);
        uint32_t u = 0;  // the group's maximum over the CTAs that hold its channels
        const int k0 = of * a.G / g.cpc, k1 = (min((of + 1) * a.G, a.C) - 1) / g.cpc;
        if (k0 == k1) u = mx[gl * slots + to];
        else
          for (int z = k0; z <= k1; ++z) u = max(u, peer_load(peer(mx, z) + ((of - z * g.cpc / a.G) * slots + to) * 4));
        const float t = fmaxf(__uint_as_float(u), kAmaxFloor);
        ginv[gl * slots + to] = kE4m3Max / t;
        if (of * a.G >= first_c) a.scale[(at.b * a.NG + of) * a.P + at.pos + px] = t / kE4m3Max;  // its first CTA
      }
      __syncthreads();
      F<V> inv = fill<V>(0.0f);
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        if (i < nc && (i == 0 || grp[i] != grp[i - (i > 0)])) inv = J.get(ginv + (grp[i] - g0) * slots, m);
        lane.write(a.q, at, m, i, packed_e4m3<V>(mul(v[i], inv)), n);
      }
      // the other half is read no more (every CTA is past the last tile's
      // reads at this tile's barriers): clear it for the next tile
      uint32_t* z = gm + (parity ^ 1) * gm_half;
      for (int k = threadIdx.x; k < gm_half; k += NT) z[k] = 0u;
    }
  }
  if (Q == kAtomicQ && g.CL > 1) cluster_barrier();  // peers may still read this CTA's maxima
}

template <int Q, typename T, int NCH, bool SHIFT>
int launch_norm_tile(const NormArgs& a, const Tiling& g, int ng_max, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  using Join = Joiner<V, 1, 1, SHIFT>;
  const size_t ring = Lane<T, V, NCH, SHIFT>::words(g) * 16 * 2, slots = Join::slots_of(g);
  const size_t qb = Q == kRowsQ ? 4 * ((size_t)(g.NT / g.LX) + ng_max) * slots : Q == kAtomicQ ? 12 * ng_max * slots : 0;
  const size_t smem = ring + 4 * Join::floats(g) + qb;
  if (smem > kMaxSmem) return DISCO_ERR_UNSUPPORTED;
  return launch_clusters(norm_tile_kernel<T, NCH, Q, SHIFT>, g, smem, st, "norm_tile_kernel", a, g, ng_max);
}

template <int Q, typename T>
int norm_tile(const NormArgs& a, const Tiling& g, int ng_max, cudaStream_t st) {
  if (g.shifted)
    return g.NCH == 4 ? launch_norm_tile<Q, T, 4, true>(a, g, ng_max, st) : launch_norm_tile<Q, T, 8, true>(a, g, ng_max, st);
  return g.NCH == 4 ? launch_norm_tile<Q, T, 4, false>(a, g, ng_max, st) : launch_norm_tile<Q, T, 8, false>(a, g, ng_max, st);
}

}  // namespace norm
}  // namespace disco
