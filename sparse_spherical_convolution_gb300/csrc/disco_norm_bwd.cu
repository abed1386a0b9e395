// disco_norm_bwd.cu -- gradient of the channel norm (disco_rms_norm_bwd).
//
// With r = 1 / sqrt(mean_c h^2 + eps), n = h r and g = weight dy:
//   dx = r (g - n mean_c(g n)) + dh = (r g) - h k + dh,  k = r^3 mean_c(g h)
//   dweight[c] = sum over pixels of dy h r
// One pass over dy, h and dh; dweight leaves as one row of fp32 partial sums
// for each cluster of CTAs, summed in a fixed order by a second kernel that may
// start while the first ends.
//
// Measured (both kernels, GB300): [1,512,360x720] bf16 with dh 196 us, 5.4 TB/s
// (80 % of the copy rate); [2,128,361x720] 88 us, 6.0 TB/s; [20,64,65344] 105 us,
// the same with odd rows 149 us; [3,91,151250] (odd rows) 94 us, 3.5 TB/s.  HBM
// bounds up to 256 channels.  At 512 one CTA
// holds rows of 64 bytes, or a pair rows of 128 bytes and a cluster barrier a tile:
// 198 and 228 us.  Odd rows are bound by instructions (two sums and two factors a
// pixel to realign, 16 shared-memory accesses each way).

#include "disco_norm.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_bwd_bounds)

namespace {

using namespace norm;

constexpr int kGenParts = 304;  // rows of partial sums of the general kernel: its CTAs

// Any shape; the inputs are read again for the second pass.  A channel's sum over
// pixels stands in this CTA's row of partial sums.
template <typename T, bool ROW>
__global__ void __launch_bounds__(kGenWarps * 32) norm_bwd_any_kernel(const NormBwdArgs a, const long long tiles) {
  using D = Dealt<ROW>;
  __shared__ float buf[kGenWarps][32];
  const T *dy = (const T*)a.dy, *h = (const T*)a.h, *w = (const T*)a.w, *dh = (const T*)a.dh;
  T* dx = (T*)a.dx;
  const long long tpb = (a.P + D::PX - 1) / D::PX;
  float* part = a.part ? a.part + (long long)blockIdx.x * a.C : nullptr;
  const bool owner = D::pixel() == 0;  // of its channels' sums
  if (part && owner)
    for (int c = D::first(); c < a.C; c += D::STEP) part[c] = 0.0f;
  auto plus = [](float u, float v) { return u + v; };
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const long long b = t / tpb, p = (t - b * tpb) * D::PX + D::pixel();
    const bool live = p < a.P;
    const long long base = b * a.C * a.P + p;
    float s = 0.0f, d = 0.0f;
    if (live)
      for (int c = D::first(); c < a.C; c += D::STEP) {
        const long long i = base + c * a.P;
        const float v = to_f32(h[i]);
        s = fmaf(v, v, s);
        d = fmaf(to_f32(dy[i]) * (w ? to_f32(w[c]) : 1.0f), v, d);
      }
    const float r = 1.0f / sqrtf(D::join(s, buf, plus) / (float)a.C + a.eps);
    const float k = D::join(d, buf, plus) * r / (float)a.C;  // mean_c(g n)
    for (int c = D::first(); c < a.C; c += D::STEP) {
      const long long i = base + c * a.P;
      float u = 0.0f;
      if (live) {
        const float n = to_f32(h[i]) * r, g = to_f32(dy[i]);
        float o = r * (g * (w ? to_f32(w[c]) : 1.0f) - n * k);
        if (dh) o += to_f32(dh[i]);
        dx[i] = from_f32<T>(o);
        u = g * n;
      }
      if (part) {
        if (!ROW)
          for (int m = 16; m; m >>= 1) u += __shfl_xor_sync(0xffffffffu, u, m);
        if (owner) part[c] += u;
      }
    }
  }
}

// Tiles (disco_norm.cuh).  A thread keeps its dy and h as loaded, in registers,
// while its shared memory takes in those of the next tile; dh waits in shared
// memory until the outputs need it.  dweight is summed in registers over all
// tiles of the CTA: its channels stay the same.
template <typename T, bool SHIFT>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_tile_kernel(const NormBwdArgs a, const Tiling g) {
  constexpr int V = 16 / (int)sizeof(T), NCH = 4;
  using L = Lane<T, V, NCH, SHIFT>;
  using W = typename L::W;
  using Join = Joiner<V, 2, 2, SHIFT>;
  extern __shared__ __align__(16) char smem[];
  if (a.part) let_next_begin();
  const uint32_t rank = g.CL > 1 ? cluster_rank() : 0;
  float* fsm = (float*)(smem + L::words(g) * 16 * (a.dh ? 3 : 2));
  const Join J(g, fsm, rank);
  const L lane(g, a.B, a.C, a.P, J.lx, J.j, (int)rank * g.cpc, smem);
  const int nc = lane.nc;
  const T *dy = (const T*)a.dy, *h = (const T*)a.h, *w = (const T*)a.w, *dh = (const T*)a.dh;
  W *r_dy = lane.slot, *r_h = r_dy + L::words(g), *r_dh = r_h + L::words(g);

  float wt[NCH], dw[NCH][2];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    wt[i] = i < nc && w ? to_f32(w[lane.channel(i)]) : 1.0f;
    dw[i][0] = dw[i][1] = 0.0f;
    if (i >= nc) {  // channels past the last: zeros, never copied over
      memset(r_dy + i * lane.stride, 0, 16);
      memset(r_h + i * lane.stride, 0, 16);
    }
  }

  Cursor at(g, a.C, a.P, blockIdx.x / g.CL), ahead = at;
  lane.fetch(g, at, dy, r_dy);
  lane.fetch(g, at, h, r_h);
  copy_commit();
  if (dh) lane.fetch(g, at, dh, r_dh);
  copy_commit();
  if (g.CL > 1) cluster_barrier();  // every CTA runs before another writes its shared memory

  for (int parity = 0; at.t < g.tiles; at = ahead, parity ^= 1) {
    const int n = (int)min((long long)g.TP, a.P - at.pos), m = lane.skew(at);  // n: pixels of the tile
    ahead.next(g);
    W k_dy[NCH], k_h[NCH];
    copy_wait<1>();  // all but dh
    uint4 mask;
    if (SHIFT) mask = lane.mask(m, n);
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      k_dy[i] = lane.read(r_dy, i);
      k_h[i] = lane.read(r_h, i);
      if (SHIFT) k_dy[i] = k_dy[i] & mask, k_h[i] = k_h[i] & mask;
    }
    lane.fetch(g, ahead, dy, r_dy);
    lane.fetch(g, ahead, h, r_h);
    copy_commit();
    F<V> s[2] = {fill<V>(0.0f), fill<V>(0.0f)}, rk[2];  // sum h^2 and sum g h; r and -r^3 mean(g h)
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const F<V> vh = unpack<T, V>(k_h[i]);
      s[0] = fma(vh, vh, s[0]);
      s[1] = fma(mul(unpack<T, V>(k_dy[i]), fill<V>(wt[i])), vh, s[1]);
    }
    auto finish = [&](const float(&z)[2], float(&out)[2]) {
      const float r = inverse_rms(z[0], a.inv_C, a.eps);
      out[0] = r;
      out[1] = -(z[1] * a.inv_C * r) * r * r;
    };
    J.submit(s, m, parity, finish);
    J.collect(rk, m, parity, finish);
    if (SHIFT)  // no statistics where there are no pixels
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (!lane.in(e, m, n)) rk[0].v[e] = rk[1].v[e] = 0.0f;
    copy_wait<1>();  // this tile's dh; the next dy and h may be on their way
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const F<V> vh = unpack<T, V>(k_h[i]), rg = mul(unpack<T, V>(k_dy[i]), rk[0]);
      F<V> d = mul(vh, rk[1]);
      if (dh) d = add(d, unpack<T, V>(lane.read(r_dh, i)));
      d = fma(rg, fill<V>(wt[i]), d);
      lane.write(a.dx, at, m, i, packed<T, V>(d), n);
      if (SHIFT || J.lx * V < n) {
        F<2> t{dw[i][0], dw[i][1]};
#pragma unroll
        for (int e = 0; e < V; e += 2) t = fma(F<2>{rg.v[e], rg.v[e + 1]}, F<2>{vh.v[e], vh.v[e + 1]}, t);
        dw[i][0] = t.v[0], dw[i][1] = t.v[1];
      }
    }
    if (dh) lane.fetch(g, ahead, dh, r_dh);
    copy_commit();
  }

  // this cluster's sums over pixels
  if (!a.part) return;
  float* row = a.part + (long long)(blockIdx.x / g.CL) * a.C;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float z = dw[i][0] + dw[i][1];
    for (int m = g.LX / 2; m; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
    if (J.lx == 0 && i < nc) row[lane.channel(i)] = z;
  }
}

// dweight[c]: the rows of partial sums, 32 threads to a channel, all of a
// thread's loads in flight (up to 10 rows: 304 CTAs).
template <typename T>
__global__ void __launch_bounds__(1024) norm_dweight_kernel(const float* part, T* dw, int parts, int C) {
  __shared__ float buf[32][33];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  wait_for_previous();
  if (c < C)
#pragma unroll 10
    for (int i = k; i < parts; i += 32) s += part[(long long)i * C + c];
  buf[k][lane] = s;
  __syncthreads();
  s = buf[lane][k];  // channel k of this CTA
#pragma unroll
  for (int m = 16; m; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
  if (lane == 0 && blockIdx.x * 32 + k < C) dw[blockIdx.x * 32 + k] = from_f32<T>(s);
}

// Rows of partial sums of a call.
int bwd_parts(int B, int C, long long P, int es) {
  Tiling g;
  if (P == 1) {
    const int rows = norm_bwd_rows_parts(B, C, es);
    if (rows) return rows;
  } else if (plan_tiles(B, C, P, es, false, &g)) return g.clusters;
  return (int)min((long long)kGenParts, (long long)B * ((P + 31) / 32));
}

template <typename T, bool SHIFT>
int launch_bwd_tile(const NormBwdArgs& a, const Tiling& g, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const size_t smem = Lane<T, V, 4, SHIFT>::words(g) * 16 * (a.dh ? 3 : 2) + 4 * Joiner<V, 2, 2, SHIFT>::floats(g);
  return launch_clusters(norm_bwd_tile_kernel<T, SHIFT>, g, smem, st, "norm_bwd_tile_kernel", a, g);
}

template <typename T>
int bwd_main(const NormBwdArgs& a, cudaStream_t st) {
  Tiling g;
  const int es = (int)sizeof(T);
  if (a.P > 1 && plan_tiles(a.B, a.C, a.P, es, false, &g))
    return g.shifted ? launch_bwd_tile<T, true>(a, g, st) : launch_bwd_tile<T, false>(a, g, st);
  const int grid = bwd_parts(a.B, a.C, a.P, es);
  const long long tiles = (long long)a.B * ((a.P + 31) / 32);
  if (a.P == 1) norm_bwd_any_kernel<T, true><<<grid, kGenWarps * 32, 0, st>>>(a, tiles);
  else norm_bwd_any_kernel<T, false><<<grid, kGenWarps * 32, 0, st>>>(a, tiles);
  return check_launch("norm_bwd_any_kernel");
}

}  // namespace
}  // namespace disco

using namespace disco;
using namespace disco::norm;

extern "C" size_t disco_rms_norm_bwd_workspace_bytes(int32_t B, int32_t C, int64_t P, disco_dtype dtype) {
  if (check_shape(B, C, P, dtype)) return 0;
  return (size_t)bwd_parts(B, C, P, elem_bytes(dtype)) * C * sizeof(float);
}

extern "C" int disco_rms_norm_bwd(const void* dy, const void* h, const void* weight, const void* dh, float eps,
                                  void* dx, void* dweight, int32_t B, int32_t C, int64_t P, disco_dtype dtype,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  disco::NvtxScope nvtx_scope("disco_rms_norm_bwd");
  int rc;
  if ((rc = check_shape(B, C, P, dtype)) || (rc = check_eps(eps))) return rc;
  if (!dy || !h || !dx) return fail(DISCO_ERR_INVALID_ARG, "dy, h or dx is null");
  const size_t need = disco_rms_norm_bwd_workspace_bytes(B, C, P, dtype);
  if (dweight && (!workspace || workspace_bytes < need))
    return fail(DISCO_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if ((rc = check_device())) return rc;
  const size_t n = (size_t)B * C * P, e = elem_bytes(dtype);
  const Buffer in[] = {{dy, n * e, "dy"}, {h, n * e, "h"}, {weight, C * e, "weight"}, {dh, n * e, "dh"}};
  const Buffer out[] = {{dx, n * e, "dx"}, {dweight, C * e, "dweight"}, {dweight ? workspace : nullptr, need, "workspace"}};
  const unsigned in_place[] = {1, 1, 0, 1};
  if ((rc = check_buffers(in, in_place, 4, out, 3))) return rc;
  const NormBwdArgs a{dy, h, weight, dh, dx, dweight ? (float*)workspace : nullptr, eps, 1.0f / (float)C, B, C, P};
  const cudaStream_t st = (cudaStream_t)stream;
  rc = P == 1 ? norm_bwd_by_rows(a, dtype, st) : DISCO_ERR_UNSUPPORTED;
  if (rc == DISCO_ERR_UNSUPPORTED) {
#define CALL(T) rc = bwd_main<T>(a, st)
    DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  }
  if (rc || !dweight) return rc;
  const int parts = (int)(need / ((size_t)C * sizeof(float)));
#define CALL(T) \
  rc = launch(norm_dweight_kernel<T>, (C + 31) / 32, 1024, 1, true, 0, 0, st, "norm_dweight_kernel", (const float*)a.part, (T*)dweight, parts, C)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}
