// disco_norm.cu -- channel RMS norm with the residual's addition and an
// 8-bit copy (disco_rms_norm), its gradient (disco_rms_norm_bwd) and the
// return from 8 bits (disco_dequant_e4m3), on activations [B, C, P].
//
// The general kernels below take every shape: 32 pixels per CTA, the channels
// dealt to 8 warps, statistics joined in shared memory, the inputs read again
// for each further pass.

#include "disco_norm.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_bounds)

namespace {

using namespace norm;

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;  // group maximum of an all-zero group: its scale stays above 0
constexpr int kGenWarps = 8;

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float from_e4m3(uint8_t v) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)v, __NV_E4M3)));
}

struct NormArgs {
  const void *x, *res, *w;
  void *h, *y, *q;
  float* scale;
  float eps, inv_C;
  int G, NG, ng_max, B, C;  // ng_max: groups that touch one CTA's channels
  long long P, tiles;       // tiles: of the general kernel
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
__device__ __forceinline__ float warps_max(float v, float (*buf)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  buf[warp][lane] = v;
  __syncthreads();
  float s = 0.0f;
  for (int i = 0; i < kGenWarps; ++i) s = fmaxf(s, buf[i][lane]);
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kGenWarps * 32) norm_any_kernel(const NormArgs a) {
  __shared__ float buf[kGenWarps][32];
  const T *x = (const T*)a.x, *res = (const T*)a.res, *w = (const T*)a.w;
  T *h = (T*)a.h, *y = (T*)a.y;
  uint8_t* q = (uint8_t*)a.q;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long tpb = (a.P + 31) / 32;
  for (long long t = blockIdx.x; t < a.tiles; t += gridDim.x) {
    const long long b = t / tpb, p = (t - b * tpb) * 32 + lane;
    const bool live = p < a.P;
    const long long base = b * a.C * a.P + p;
    auto value = [&](int c) {
      const long long i = base + c * a.P;
      float v = to_f32(x[i]);
      return res ? v + to_f32(res[i]) : v;
    };
    float s = 0.0f;
    if (live)
      for (int c = warp; c < a.C; c += kGenWarps) {
        const float v = value(c);
        s = fmaf(v, v, s);
      }
    const float r = 1.0f / sqrtf(warps_sum(s, buf) / (float)a.C + a.eps);
    for (int g = 0; g < a.NG; ++g) {
      const int c0 = g * a.G, c1 = min(a.C, c0 + a.G);
      float inv = 0.0f;
      if (q) {
        float m = 0.0f;
        if (live)
          for (int c = c0 + warp; c < c1; c += kGenWarps) {
            const float v = value(c) * r * (w ? to_f32(w[c]) : 1.0f);
            m = fmaxf(m, fabsf(v));
          }
        m = fmaxf(warps_max(m, buf), kAmaxFloor);
        inv = kE4m3Max / m;
        if (live && warp == 0) a.scale[(b * a.NG + g) * a.P + p] = m / kE4m3Max;
      }
      if (live)
        for (int c = c0 + warp; c < c1; c += kGenWarps) {
          const long long i = base + c * a.P;
          const float v = value(c), n = v * r * (w ? to_f32(w[c]) : 1.0f);
          if (h) h[i] = from_f32<T>(v);
          if (y) y[i] = from_f32<T>(n);
          if (q) q[i] = to_e4m3(n * inv);
        }
    }
  }
}


// ---- tiles: one pass over the data ----------------------------------------
//
// Bound by HBM.  Every input is read once and held: a thread's V x NCH sums
// x + residual stay in fp32 registers between the statistics and the outputs,
// so y is computed from the unrounded h, while its shared memory already takes
// in the next tile (thread-private cp.async).

template <typename T, int V, int NCH, bool Q>
__global__ void __launch_bounds__(kMaxThreads) norm_tile_kernel(const NormArgs a, const Tiling g) {
  constexpr int VB = V * (int)sizeof(T);
  constexpr bool kAsync = VB >= 4;  // cp.async copies 4, 8 or 16 bytes
  using W = Raw<T, V>;
  extern __shared__ __align__(16) char smem[];
  const uint32_t rank = g.CL > 1 ? cluster_rank() : 0;
  const int streams = a.res ? 2 : 1;
  W* ring = (W*)smem;
  float* fsm = (float*)(smem + (kAsync ? (size_t)g.NT * NCH * VB * streams : 0));
  const Joiner<V, 1> J(g, fsm, rank);
  const int NT = g.NT, TP = J.TP;
  const int c0 = (int)rank * g.cpc + J.j * NCH;
  const int nc = max(0, min(min((int)(rank + 1) * g.cpc, a.C) - c0, NCH));
  const T *x = (const T*)a.x, *res = (const T*)a.res, *w = (const T*)a.w;
  T *h = (T*)a.h, *y = (T*)a.y;
  W *rx = ring + threadIdx.x, *rr = rx + NT * NCH;
  [[maybe_unused]] const long long total = (long long)a.B * a.C * a.P;  // for the range checks

  float wt[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    wt[i] = i < nc && w ? to_f32(w[c0 + i]) : 1.0f;
    if (kAsync && i >= nc) {  // channels past the last: zeros, never copied over
      memset(rx + i * NT, 0, VB);
      if (res) memset(rr + i * NT, 0, VB);
    }
  }
  // 8-bit copy: this CTA's groups g0 .. g0 + ng - 1, their maxima of the two
  // last tiles in turn
  const int first_c = (int)rank * g.cpc, last_c = min(first_c + g.cpc, a.C) - 1;
  const int g0 = Q ? first_c / a.G : 0, ng = Q && last_c >= first_c ? last_c / a.G - g0 + 1 : 0;
  uint32_t* gm = (uint32_t*)(fsm + Joiner<V, 1>::floats(g));
  const int gm_half = a.ng_max * TP;
  if (Q)
    for (int k = threadIdx.x; k < 2 * gm_half; k += NT) gm[k] = 0u;

  Cursor at(g, blockIdx.x / g.CL), ahead = at;
  auto offset = [&](const Cursor& c) { return (c.b * a.C + c0) * a.P + c.ti * TP + J.lx * V; };
  auto live = [&](const Cursor& c) { return c.t < g.tiles && c.ti * TP + J.lx * V < a.P; };
  auto fetch = [&]() {
    if (live(ahead)) {
      const long long o = offset(ahead);
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc && DISCO_IN_BOUNDS(o + i * a.P >= 0 && o + i * a.P + V <= total)) {
          copy_async<kAsync ? VB : 4>(rx + i * NT, x + o + i * a.P);
          if (res) copy_async<kAsync ? VB : 4>(rr + i * NT, res + o + i * a.P);
        }
    }
    copy_commit();
    ahead.next(g);
  };
  if (kAsync) fetch();
  if (g.CL > 1) cluster_barrier();  // every CTA runs before another writes its shared memory

  for (int parity = 0; at.t < g.tiles; at.next(g), parity ^= 1) {
    const long long o = offset(at);
    const bool on = live(at);
    F<V> v[NCH];
    if constexpr (kAsync) {
      copy_wait<0>();
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        v[i] = unpack<T, V>(rx[i * NT]);
        if (res) v[i] = add(v[i], unpack<T, V>(rr[i * NT]));
      }
      fetch();
    } else {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        v[i] = fill<V>(0.0f);
        if (on && i < nc && DISCO_IN_BOUNDS(o + i * a.P >= 0 && o + i * a.P + V <= total)) {
          v[i] = unpack<T, V>(load_stream<W>(x + o + i * a.P));
          if (res) v[i] = add(v[i], unpack<T, V>(load_stream<W>(res + o + i * a.P)));
        }
      }
    }
    F<V> s[1] = {fill<V>(0.0f)};
#pragma unroll
    for (int i = 0; i < NCH; ++i) s[0] = fma(v[i], v[i], s[0]);
    if (h && on)
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc && DISCO_IN_BOUNDS(o + i * a.P + V <= total)) store_stream(h + o + i * a.P, packed<T, V>(v[i]));
    J.join(s, parity);
    F<V> r;
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = rsqrtf(fmaf(s[0].v[e], a.inv_C, a.eps));
#pragma unroll
    for (int i = 0; i < NCH; ++i) v[i] = mul(mul(v[i], r), fill<V>(wt[i]));
    if (y && on)
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc && DISCO_IN_BOUNDS(o + i * a.P + V <= total)) store_stream(y + o + i * a.P, packed<T, V>(v[i]));
    if constexpr (Q) {
      uint32_t* m = gm + parity * gm_half;
      if (nc > 0) {
        int grp = c0 / a.G, left = (grp + 1) * a.G - c0;  // channels to the group's end
        F<V> top = fill<V>(0.0f);
#pragma unroll
        for (int i = 0; i < NCH; ++i)
          if (i < nc) {
#pragma unroll
            for (int e = 0; e < V; ++e) top.v[e] = fmaxf(top.v[e], fabsf(v[i].v[e]));  // a NaN does not count
            if (--left == 0 || i == nc - 1) {
#pragma unroll
              for (int e = 0; e < V; ++e) atomicMax(m + (grp - g0) * TP + J.lx * V + e, __float_as_uint(top.v[e]));
              top = fill<V>(0.0f);
              ++grp;
              left = a.G;
            }
          }
      }
      if (g.CL > 1) cluster_barrier();
      else __syncthreads();
      // a group's maximum over the CTAs that hold its channels
      auto maximum = [&](int grp, int px) {
        uint32_t u = 0;
        const int k0 = grp * a.G / g.cpc, k1 = (min((grp + 1) * a.G, a.C) - 1) / g.cpc;
        if (k0 == k1) u = m[(grp - g0) * TP + px];
        else
          for (int k = k0; k <= k1; ++k)
            u = max(u, peer_load(peer(m, k) + ((grp - k * g.cpc / a.G) * TP + px) * 4));
        return fmaxf(__uint_as_float(u), kAmaxFloor);
      };
      if (on && nc > 0) {
        int grp = c0 / a.G, left = 0;
        F<V> inv;
        uint8_t* q = (uint8_t*)a.q;
#pragma unroll
        for (int i = 0; i < NCH; ++i)
          if (i < nc) {
            if (left == 0) {
              if (i > 0) ++grp;
              left = i > 0 ? a.G : (grp + 1) * a.G - c0;
#pragma unroll
              for (int e = 0; e < V; ++e) inv.v[e] = kE4m3Max / maximum(grp, J.lx * V + e);
            }
            --left;
            if (DISCO_IN_BOUNDS(o + i * a.P + V <= total))
              store_stream(q + o + i * a.P, packed_e4m3<V>(mul(v[i], inv)));
          }
      }
      // scales of the groups that begin in this CTA
      for (int k = threadIdx.x; k < ng * TP; k += NT) {
        const int gl = k / TP, px = k - gl * TP, grp = g0 + gl;
        const long long p = at.ti * TP + px;
        if (p < a.P && grp * a.G >= first_c) a.scale[(at.b * a.NG + grp) * a.P + p] = maximum(grp, px) / kE4m3Max;
      }
      // the other half is read no more (every CTA is past the last tile's
      // reads at this tile's barriers): clear it for the next tile
      uint32_t* z = gm + (parity ^ 1) * gm_half;
      for (int k = threadIdx.x; k < gm_half; k += NT) z[k] = 0u;
    }
  }
  if (Q && g.CL > 1) cluster_barrier();  // peers may still read this CTA's maxima
}

// Bytes of shared memory of a launch.
template <int V>
size_t norm_tile_smem(const NormArgs& a, const Tiling& g, int es, bool q) {
  const int VB = V * es;
  return (VB >= 4 ? (size_t)g.NT * g.NCH * VB * (a.res ? 2 : 1) : 0) + 4 * Joiner<V, 1>::floats(g) +
         (q ? 8 * (size_t)a.ng_max * g.LX * V : 0);
}

template <typename T, int V, int NCH>
int norm_tile(const NormArgs& a, const Tiling& g, size_t smem, cudaStream_t st) {
  return a.q ? launch_clusters(norm_tile_kernel<T, V, NCH, true>, g, smem, st, "norm_tile_kernel", a, g)
             : launch_clusters(norm_tile_kernel<T, V, NCH, false>, g, smem, st, "norm_tile_kernel", a, g);
}

// DISCO_ERR_UNSUPPORTED, without launching, for shapes the tiles do not take.
template <typename T>
int norm_by_tiles(NormArgs& a, cudaStream_t st) {
  Tiling g;
  if (!plan_tiles(a.B, a.C, a.P, (int)sizeof(T), 2, &g)) return DISCO_ERR_UNSUPPORTED;
  a.ng_max = a.q ? min(a.NG, (g.cpc + a.G - 1) / a.G + 1) : 0;
  constexpr int VM = 16 / (int)sizeof(T);
  const size_t smem = g.V == VM ? norm_tile_smem<VM>(a, g, sizeof(T), a.q)
                      : g.V == 2 ? norm_tile_smem<2>(a, g, sizeof(T), a.q)
                                 : norm_tile_smem<1>(a, g, sizeof(T), a.q);
  if (smem > kMaxSmem) return DISCO_ERR_UNSUPPORTED;
  if (g.V == VM) return g.NCH == 4 ? norm_tile<T, VM, 4>(a, g, smem, st) : norm_tile<T, VM, 8>(a, g, smem, st);
  if constexpr (sizeof(T) == 2)
    if (g.V == 2) return g.NCH == 8 ? norm_tile<T, 2, 8>(a, g, smem, st) : norm_tile<T, 2, 16>(a, g, smem, st);
  return g.NCH == 8 ? norm_tile<T, 1, 8>(a, g, smem, st) : norm_tile<T, 1, 16>(a, g, smem, st);
}

struct DequantArgs {
  const uint8_t* q;
  const float* scale;
  void* x;
  int G, NG, C;
  long long P, n;
};

template <typename T>
__global__ void dequant_any_kernel(const DequantArgs a) {
  T* x = (T*)a.x;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < a.n; i += (long long)gridDim.x * blockDim.x) {
    const long long bc = i / a.P, p = i - bc * a.P, b = bc / a.C;
    const int c = (int)(bc - b * a.C);
    x[i] = from_f32<T>(from_e4m3(a.q[i]) * a.scale[(b * a.NG + c / a.G) * a.P + p]);
  }
}

int groups(int32_t C, int32_t group, int* G) {
  *G = group > 0 && group < C ? group : C;
  return (C + *G - 1) / *G;
}

}  // namespace

namespace norm {

namespace {
bool overlap(const Buffer& u, const Buffer& v) {
  const char *a = (const char*)u.p, *b = (const char*)v.p;
  return u.p && v.p && a < b + v.bytes && b < a + u.bytes;
}
}  // namespace

// Device memory, alignment, and no output over another buffer but for in
// place pairs (in_place[i] bit o: input i may be output o).
int check_buffers(const Buffer* in, const unsigned* in_place, int nin, const Buffer* out, int nout) {
  int rc;
  for (int k = 0; k < nin + nout; ++k) {
    const Buffer& u = k < nin ? in[k] : out[k - nin];
    if (!u.p) continue;
    if (!aligned16(u.p)) return fail(DISCO_ERR_ALIGNMENT, "%s must be 16-byte aligned", u.name);
    if ((rc = check_dev_ptr(u.p, u.name))) return rc;
  }
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i)
      if (overlap(out[o], in[i]) && !((in_place[i] >> o & 1u) && out[o].p == in[i].p))
        return fail(DISCO_ERR_INVALID_ARG, "%s overlaps %s", out[o].name, in[i].name);
    for (int j = 0; j < o; ++j)
      if (overlap(out[o], out[j])) return fail(DISCO_ERR_INVALID_ARG, "%s overlaps %s", out[o].name, out[j].name);
  }
  return DISCO_OK;
}

int check_shape(int32_t B, int32_t C, int64_t P, disco_dtype dtype) {
  if (dtype != DISCO_F32 && dtype != DISCO_BF16 && dtype != DISCO_F16) return fail(DISCO_ERR_UNSUPPORTED, "dtype");
  if (B < 1 || C < 1 || P < 1) return fail(DISCO_ERR_INVALID_ARG, "B, C and P must be >= 1");
  if (C > 1 << 30) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^30 channels");
  if ((double)B * C * (double)P > 1e15) return fail(DISCO_ERR_UNSUPPORTED, "more than 1e15 elements");
  return DISCO_OK;
}

int check_eps(float eps) {
  if (!(eps > 0.0f) || isinf(eps)) return fail(DISCO_ERR_INVALID_ARG, "eps must be positive and finite");
  return DISCO_OK;
}

bool plan_tiles(int B, int C, long long P, int es, int most, Tiling* g) {
  g->V = es == 4 ? (P % 4 == 0 ? 4 : 1) : (P % 8 == 0 ? 8 : P % 2 == 0 ? 2 : 1);
  const bool wide = g->V * es == 16;
  const int few = wide ? 4 : 8, many = most * few;
  const long long vecs = P / g->V;
  int LX = wide ? 16 : g->V * es == 4 ? 32 : 64;
  while (LX > 1 && LX / 2 >= vecs) LX /= 2;
  // fewer pixels to a tile while there are not two tiles for each SM
  while (LX > 4 && (long long)B * ((vecs + LX - 1) / LX) < 2 * kSMs) LX /= 2;
  for (;; LX /= 2) {
    bool done = false;
    for (int CL = 1; CL <= 8 && !done; CL *= 2)
      for (int NCH = few; NCH <= many && !done; NCH *= 2) {
        const int cpc = (C + CL - 1) / CL, NL = (cpc + NCH - 1) / NCH;
        const int NT = (LX * NL + 31) / 32 * 32;
        if (NT > kMaxThreads) continue;
        g->CL = CL, g->NCH = NCH, g->cpc = cpc, g->NT = NT, g->LX = LX;
        done = true;
      }
    if (done) break;
    if (LX == 1) return false;
  }
  g->tpb = (vecs + g->LX - 1) / g->LX;
  g->tiles = B * g->tpb;
  const int per_sm = max(1, kMaxThreads / g->NT);
  const long long clusters = max(1, kSMs * per_sm / g->CL);
  g->clusters = (int)min(g->tiles, clusters);
  g->step_b = g->clusters / g->tpb;
  g->step_t = g->clusters % g->tpb;
  return true;
}

}  // namespace norm
}  // namespace disco

using namespace disco;
using namespace disco::norm;

extern "C" int disco_rms_norm(const void* x, const void* residual, const void* weight, float eps, void* h, void* y,
                              void* q, float* scale, int32_t group, int32_t B, int32_t C, int64_t P,
                              disco_dtype dtype, void* stream) {
  disco::NvtxScope nvtx_scope("disco_rms_norm");
  int rc;
  if ((rc = check_shape(B, C, P, dtype)) || (rc = check_eps(eps))) return rc;
  if (!x) return fail(DISCO_ERR_INVALID_ARG, "x is null");
  if (!y && !q) return fail(DISCO_ERR_INVALID_ARG, "neither y nor q is given");
  if (!q != !scale) return fail(DISCO_ERR_INVALID_ARG, "q and scale come together");
  if (h && !residual) return fail(DISCO_ERR_INVALID_ARG, "h without a residual is x itself");
  if (group < 0) return fail(DISCO_ERR_INVALID_ARG, "group must be >= 0");
  if ((rc = check_device())) return rc;
  NormArgs a{x, residual, weight, h, y, q, scale, eps, 1.0f / (float)C, 0, 0, 0, B, C, P, (long long)B * ((P + 31) / 32)};
  a.NG = groups(C, group, &a.G);
  if (!q) a.G = C, a.NG = 1;
  const size_t n = (size_t)B * C * P, e = elem_bytes(dtype);
  const Buffer in[] = {{x, n * e, "x"}, {residual, n * e, "residual"}, {weight, C * e, "weight"}};
  const Buffer out[] = {{h, n * e, "h"}, {y, n * e, "y"}, {q, n, "q"}, {scale, (size_t)B * a.NG * P * 4, "scale"}};
  const unsigned in_place[] = {3, 3, 0};
  if ((rc = check_buffers(in, in_place, 3, out, 4))) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
#define CALL(T) rc = norm_by_tiles<T>(a, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  if (rc != DISCO_ERR_UNSUPPORTED) return rc;
  const int grid = (int)min(a.tiles, 152LL * 8);
#define CALL(T) norm_any_kernel<T><<<grid, kGenWarps * 32, 0, st>>>(a)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("norm_any_kernel");
}

extern "C" int disco_dequant_e4m3(const void* q, const float* scale, void* x, int32_t group, int32_t B, int32_t C,
                                  int64_t P, disco_dtype dtype, void* stream) {
  disco::NvtxScope nvtx_scope("disco_dequant_e4m3");
  int rc;
  if ((rc = check_shape(B, C, P, dtype))) return rc;
  if (!q || !scale || !x) return fail(DISCO_ERR_INVALID_ARG, "q, scale or x is null");
  if (group < 0) return fail(DISCO_ERR_INVALID_ARG, "group must be >= 0");
  if ((rc = check_device())) return rc;
  DequantArgs a{(const uint8_t*)q, scale, x, 0, 0, C, P, (long long)B * C * P};
  a.NG = groups(C, group, &a.G);
  const Buffer in[] = {{q, (size_t)a.n, "q"}, {scale, (size_t)B * a.NG * P * 4, "scale"}};
  const Buffer out[] = {{x, (size_t)a.n * elem_bytes(dtype), "x"}};
  const unsigned in_place[] = {0, 0};
  if ((rc = check_buffers(in, in_place, 2, out, 1))) return rc;
  const int grid = (int)min((a.n + 255) / 256, 152LL * 8);
#define CALL(T) dequant_any_kernel<T><<<grid, 256, 0, (cudaStream_t)stream>>>(a)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("dequant_any_kernel");
}
