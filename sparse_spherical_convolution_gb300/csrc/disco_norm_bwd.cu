// disco_norm_bwd.cu -- gradient of the channel norm (disco_rms_norm_bwd).
//
// With r = 1 / sqrt(mean_c h^2 + eps), n = h r and g = weight dy:
//   dx = r (g - n mean_c(g n)) + dh = (r g) - h k + dh,  k = r^3 mean_c(g h)
//   dweight[c] = sum over pixels of dy h r
// One pass over dy, h and dh; dweight leaves as one row of fp32 partial sums
// for each cluster of CTAs, summed in a fixed order by a second kernel.

#include "disco_norm.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_bwd_bounds)

namespace {

using namespace norm;

constexpr int kGenWarps = 8;
constexpr int kGenParts = 304;  // rows of partial sums of the general kernel: its CTAs

struct NormBwdArgs {
  const void *dy, *h, *w, *dh;
  void* dx;
  float* part;
  float eps, inv_C;
  int B, C;
  long long P, tiles;  // tiles: of the general kernel
};

// sum over the 8 warps of one value per lane (pixel)
__device__ __forceinline__ float warps_sum(float v, float (*buf)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  buf[warp][lane] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kGenWarps; ++i) s += buf[i][lane];
  return s;
}

// Any shape: 32 pixels per CTA, the channels dealt to 8 warps, the inputs read
// again for the second pass.
template <typename T>
__global__ void __launch_bounds__(kGenWarps * 32) norm_bwd_any_kernel(const NormBwdArgs a) {
  __shared__ float buf[kGenWarps][32];
  const T *dy = (const T*)a.dy, *h = (const T*)a.h, *w = (const T*)a.w, *dh = (const T*)a.dh;
  T* dx = (T*)a.dx;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tpb = (a.P + 31) / 32;
  float* part = a.part ? a.part + (long long)blockIdx.x * a.C : nullptr;
  if (part)
    for (int c = warp; c < a.C; c += kGenWarps)
      if (lane == 0) part[c] = 0.0f;
  for (long long t = blockIdx.x; t < a.tiles; t += gridDim.x) {
    const long long b = t / tpb, p = (t - b * tpb) * 32 + lane;
    const bool live = p < a.P;
    const long long base = b * a.C * a.P + p;
    float s = 0.0f, d = 0.0f;
    if (live)
      for (int c = warp; c < a.C; c += kGenWarps) {
        const long long i = base + c * a.P;
        const float v = to_f32(h[i]);
        s = fmaf(v, v, s);
        d = fmaf(to_f32(dy[i]) * (w ? to_f32(w[c]) : 1.0f), v, d);
      }
    const float r = 1.0f / sqrtf(warps_sum(s, buf) / (float)a.C + a.eps);
    const float k = warps_sum(d, buf) * r / (float)a.C;  // mean_c(g n)
    for (int c = warp; c < a.C; c += kGenWarps) {
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
        for (int m = 16; m; m >>= 1) u += __shfl_xor_sync(0xffffffffu, u, m);
        if (lane == 0) part[c] += u;
      }
    }
  }
}

// Tiles (disco_norm.cuh).  A thread keeps its dy and h as loaded, in registers,
// while its shared memory takes in those of the next tile; dh waits in shared
// memory until the outputs need it.  dweight is summed in registers over all
// tiles of the CTA: its channels stay the same.
template <typename T, int V, int NCH>
__global__ void __launch_bounds__(kMaxThreads) norm_bwd_tile_kernel(const NormBwdArgs a, const Tiling g) {
  constexpr int VB = V * (int)sizeof(T);
  constexpr bool kAsync = VB >= 4;
  using W = Raw<T, V>;
  extern __shared__ __align__(16) char smem[];
  const uint32_t rank = g.CL > 1 ? cluster_rank() : 0;
  W* ring = (W*)smem;
  float* fsm = (float*)(smem + (kAsync ? (size_t)g.NT * NCH * VB * (a.dh ? 3 : 2) : 0));
  const Joiner<V, 2> J(g, fsm, rank);
  const int NT = g.NT, TP = J.TP;
  const int c0 = (int)rank * g.cpc + J.j * NCH;
  const int nc = max(0, min(min((int)(rank + 1) * g.cpc, a.C) - c0, NCH));
  const T *dy = (const T*)a.dy, *h = (const T*)a.h, *w = (const T*)a.w, *dh = (const T*)a.dh;
  T* dx = (T*)a.dx;
  W *r_dy = ring + threadIdx.x, *r_h = r_dy + NT * NCH, *r_dh = r_h + NT * NCH;
  [[maybe_unused]] const long long total = (long long)a.B * a.C * a.P;

  float wt[NCH], dw[NCH][2];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    wt[i] = i < nc && w ? to_f32(w[c0 + i]) : 1.0f;
    dw[i][0] = dw[i][1] = 0.0f;
    if (kAsync && i >= nc) {  // channels past the last: zeros, never copied over
      memset(r_dy + i * NT, 0, VB);
      memset(r_h + i * NT, 0, VB);
    }
  }

  Cursor at(g, blockIdx.x / g.CL), ahead = at;
  auto offset = [&](const Cursor& c) { return (c.b * a.C + c0) * a.P + c.ti * TP + J.lx * V; };
  auto live = [&](const Cursor& c) { return c.t < g.tiles && c.ti * TP + J.lx * V < a.P; };
  auto fetch = [&](const T* p, W* to) {
    if (live(ahead)) {
      const long long o = offset(ahead);
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc && DISCO_IN_BOUNDS(o + i * a.P >= 0 && o + i * a.P + V <= total))
          copy_async<kAsync ? VB : 4>(to + i * NT, p + o + i * a.P);
    }
  };
  if (kAsync) {
    fetch(dy, r_dy);
    fetch(h, r_h);
    copy_commit();
    if (dh) fetch(dh, r_dh);
    copy_commit();
    ahead.next(g);
  }
  if (g.CL > 1) cluster_barrier();  // every CTA runs before another writes its shared memory

  for (int parity = 0; at.t < g.tiles; at.next(g), parity ^= 1) {
    const long long o = offset(at);
    const bool on = live(at);
    W k_dy[NCH], k_h[NCH], k_dh[kAsync ? 1 : NCH];
    if constexpr (kAsync) {
      copy_wait<1>();  // all but dh
#pragma unroll
      for (int i = 0; i < NCH; ++i) k_dy[i] = r_dy[i * NT], k_h[i] = r_h[i * NT];
      fetch(dy, r_dy);
      fetch(h, r_h);
      copy_commit();
    } else {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        memset(&k_dy[i], 0, VB);
        memset(&k_h[i], 0, VB);
        if (on && i < nc && DISCO_IN_BOUNDS(o + i * a.P >= 0 && o + i * a.P + V <= total)) {
          k_dy[i] = load_stream<W>(dy + o + i * a.P);
          k_h[i] = load_stream<W>(h + o + i * a.P);
          if (dh) k_dh[i] = load_stream<W>(dh + o + i * a.P);
        }
      }
    }
    F<V> s[2] = {fill<V>(0.0f), fill<V>(0.0f)};  // sum h^2, sum g h
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const F<V> vh = unpack<T, V>(k_h[i]);
      s[0] = fma(vh, vh, s[0]);
      s[1] = fma(mul(unpack<T, V>(k_dy[i]), fill<V>(wt[i])), vh, s[1]);
    }
    J.join(s, parity);
    F<V> r, k;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      r.v[e] = rsqrtf(fmaf(s[0].v[e], a.inv_C, a.eps));
      k.v[e] = -(s[1].v[e] * a.inv_C * r.v[e]) * r.v[e] * r.v[e];
    }
    if (kAsync) copy_wait<1>();  // this tile's dh; the next dy and h may be on their way
    if (on) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc) {
          const F<V> vh = unpack<T, V>(k_h[i]), vg = unpack<T, V>(k_dy[i]);
          const F<V> rg = mul(vg, r);
          F<V> d = mul(vh, k);
          if (dh) d = add(d, unpack<T, V>(kAsync ? r_dh[i * NT] : k_dh[kAsync ? 0 : i]));
          d = fma(rg, fill<V>(wt[i]), d);
          if (DISCO_IN_BOUNDS(o + i * a.P + V <= total)) store_stream(dx + o + i * a.P, packed<T, V>(d));
          if constexpr (V % 2 == 0) {
            F<2> t{dw[i][0], dw[i][1]};
#pragma unroll
            for (int e = 0; e < V; e += 2) t = fma(F<2>{rg.v[e], rg.v[e + 1]}, F<2>{vh.v[e], vh.v[e + 1]}, t);
            dw[i][0] = t.v[0], dw[i][1] = t.v[1];
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) dw[i][0] = fmaf(rg.v[e], vh.v[e], dw[i][0]);
          }
        }
    }
    if (kAsync) {
      if (dh) fetch(dh, r_dh);
      copy_commit();
      ahead.next(g);
    }
  }

  // this cluster's sums over pixels: lanes of a warp, then the warps of a
  // channel lane (LX > 32)
  if (!a.part) return;
  float* row = a.part + (long long)(blockIdx.x / g.CL) * a.C;
  const int warps_to_lane = g.LX > 32 ? g.LX / 32 : 1;
  float* sm = J.red;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    float z = dw[i][0] + dw[i][1];
    for (int m = min(g.LX, 32) / 2; m; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
    if (g.LX <= 32) {
      if (J.lx == 0 && i < nc) row[c0 + i] = z;
    } else {
      if ((threadIdx.x & 31) == 0) sm[threadIdx.x / 32] = z;
      __syncthreads();
      if (J.lx == 0 && i < nc) {
        z = 0.0f;
        for (int k = 0; k < warps_to_lane; ++k) z += sm[threadIdx.x / 32 + k];
        row[c0 + i] = z;
      }
      __syncthreads();
    }
  }
}

// dweight[c]: the rows of partial sums, 8 threads to a channel.
template <typename T>
__global__ void __launch_bounds__(256) norm_dweight_kernel(const float* part, T* dw, int parts, int C) {
  __shared__ float buf[8][32];
  const int lane = threadIdx.x & 31, k = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < C)
#pragma unroll 8
    for (int i = k; i < parts; i += 8) s += part[(long long)i * C + c];
  buf[k][lane] = s;
  __syncthreads();
  if (k == 0 && c < C) {
    s = 0.0f;
    for (int i = 0; i < 8; ++i) s += buf[i][lane];
    dw[c] = from_f32<T>(s);
  }
}

// Channels to a thread: the fewest (dy and h stay in registers).
bool bwd_tiles(int B, int C, long long P, int es, Tiling* g) { return plan_tiles(B, C, P, es, 1, g); }

// Rows of partial sums of a call.
int bwd_parts(int B, int C, long long P, int es) {
  Tiling g;
  if (bwd_tiles(B, C, P, es, &g)) return g.clusters;
  return (int)min((long long)kGenParts, (long long)B * ((P + 31) / 32));
}

template <int V>
size_t bwd_tile_smem(const NormBwdArgs& a, const Tiling& g, int es) {
  const int VB = V * es;
  return (VB >= 4 ? (size_t)g.NT * g.NCH * VB * (a.dh ? 3 : 2) : 0) + 4 * Joiner<V, 2>::floats(g);
}

template <typename T>
int bwd_main(const NormBwdArgs& a, cudaStream_t st) {
  Tiling g;
  constexpr int es = (int)sizeof(T), VM = 16 / es;
  if (bwd_tiles(a.B, a.C, a.P, es, &g)) {
    if (g.V == VM)
      return launch_clusters(norm_bwd_tile_kernel<T, VM, 4>, g, bwd_tile_smem<VM>(a, g, es), st, "norm_bwd_tile_kernel", a, g);
    if constexpr (es == 2)
      if (g.V == 2)
        return launch_clusters(norm_bwd_tile_kernel<T, 2, 8>, g, bwd_tile_smem<2>(a, g, es), st, "norm_bwd_tile_kernel", a, g);
    return launch_clusters(norm_bwd_tile_kernel<T, 1, 8>, g, bwd_tile_smem<1>(a, g, es), st, "norm_bwd_tile_kernel", a, g);
  }
  norm_bwd_any_kernel<T><<<bwd_parts(a.B, a.C, a.P, es), kGenWarps * 32, 0, st>>>(a);
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
  const NormBwdArgs a{dy, h, weight, dh, dx, dweight ? (float*)workspace : nullptr, eps, 1.0f / (float)C, B, C, P,
                      (long long)B * ((P + 31) / 32)};
  const cudaStream_t st = (cudaStream_t)stream;
#define CALL(T) rc = bwd_main<T>(a, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  if (rc || !dweight) return rc;
  const int parts = (int)(need / ((size_t)C * sizeof(float)));
#define CALL(T) norm_dweight_kernel<T><<<(C + 31) / 32, 256, 0, st>>>(a.part, (T*)dweight, parts, C)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("norm_dweight_kernel");
}
