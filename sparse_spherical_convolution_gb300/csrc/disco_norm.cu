// disco_norm.cu -- channel RMS norm with the residual's addition and an
// 8-bit copy (disco_rms_norm), on activations [B, C, P]: checks, the choice of a
// kernel, and the general one.
//
//   h = x + residual,  y = weight h / sqrt(mean_c h^2 + eps),
//   q = e4m3(y 448 / m), scale = m / 448, m the largest |y| of a group of channels
//
// P = 1: rows of features (disco_norm_rows.cu).  Else tiles of pixels
// (disco_norm_tile.cuh).  What neither takes (rows past 32,768 16-bit or 16,384
// fp32 features, pixels whose channels fit no cluster, group maxima that fit no
// shared memory) runs the general kernel below, which takes every shape and
// reads the inputs again for each further pass.  It is bound by those reads:
// [1,512,360x720] bf16 with a residual takes it 468 us, the tiles 174.

#include "disco_norm.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_bounds)

namespace {

using namespace norm;

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return (uint8_t)__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}

template <typename T, bool ROW>
__global__ void __launch_bounds__(kGenWarps * 32) norm_any_kernel(const NormArgs a, const long long tiles) {
  using D = Dealt<ROW>;
  __shared__ float buf[kGenWarps][32];
  const T *x = (const T*)a.x, *res = (const T*)a.res, *w = (const T*)a.w;
  T *h = (T*)a.h, *y = (T*)a.y;
  uint8_t* q = (uint8_t*)a.q;
  const long long tpb = (a.P + D::PX - 1) / D::PX;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const long long b = t / tpb, p = (t - b * tpb) * D::PX + D::pixel();
    const bool live = p < a.P;
    const long long base = b * a.C * a.P + p;
    auto value = [&](int c) {
      const long long i = base + c * a.P;
      float v = to_f32(x[i]);
      return res ? v + to_f32(res[i]) : v;
    };
    float s = 0.0f;
    if (live)
      for (int c = D::first(); c < a.C; c += D::STEP) {
        const float v = value(c);
        s = fmaf(v, v, s);
      }
    s = D::join(s, buf, [](float u, float v) { return u + v; });
    const float r = 1.0f / sqrtf(s / (float)a.C + a.eps);
    for (int g = 0; g < a.NG; ++g) {
      const int c0 = g * a.G, c1 = min(a.C, c0 + a.G);
      float inv = 0.0f;
      if (q) {
        float m = 0.0f;
        if (live)
          for (int c = c0 + D::first(); c < c1; c += D::STEP) {
            const float v = value(c) * r * (w ? to_f32(w[c]) : 1.0f);
            m = fmaxf(m, fabsf(v));  // a NaN does not count
          }
        m = fmaxf(D::join(m, buf, [](float u, float v) { return fmaxf(u, v); }), kAmaxFloor);
        inv = kE4m3Max / m;
        if (live && D::first() == 0) a.scale[(b * a.NG + g) * a.P + p] = m / kE4m3Max;
      }
      if (live)
        for (int c = c0 + D::first(); c < c1; c += D::STEP) {
          const long long i = base + c * a.P;
          const float v = value(c), n = v * r * (w ? to_f32(w[c]) : 1.0f);
          if (h) h[i] = from_f32<T>(v);
          if (y) y[i] = from_f32<T>(n);
          if (q) q[i] = to_e4m3(n * inv);
        }
    }
  }
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

bool plan_tiles(int B, int C, long long P, int es, bool forward, Tiling* g) {
  g->V = 16 / es;
  g->apart = 1;
  while (P * g->apart % g->V) g->apart *= 2;
  g->shifted = g->apart > 1;
  const int spare = g->shifted ? 1 : 0;  // a row's words cover one less than their pixels
  const long long words = (P + g->V - 1) / g->V + spare;
  // Lanes of a row, channels of a thread, CTAs of a cluster, for up to so many
  // channels, in the order of preference; the first that gives the SM three
  // quarters of kMaxThreads.
  struct Shape {
    int LX, NCH, CL, most;
  };
  constexpr int kAny = 1 << 30;
  static const Shape fwd[] = {{16, 4, 1, kAny}, {8, 4, 1, kAny},  {16, 8, 1, kAny}, {8, 8, 1, 256},   {16, 8, 2, kAny}, {8, 8, 2, kAny},
                              {4, 8, 2, kAny},  {4, 8, 4, kAny},  {4, 8, 8, kAny},  {2, 8, 8, kAny},  {1, 8, 8, kAny}};
  static const Shape fwd_odd[] = {{32, 4, 1, kAny}, {16, 4, 1, kAny}, {32, 8, 1, kAny}, {16, 8, 1, kAny}, {8, 8, 1, 256}, {16, 8, 2, kAny},
                                  {8, 8, 2, kAny},  {4, 8, 2, kAny},  {4, 8, 4, kAny},  {4, 8, 8, kAny},  {2, 8, 8, kAny}};
  static const Shape bwd[] = {{16, 4, 1, kAny}, {8, 4, 1, kAny}, {4, 4, 1, kAny}, {4, 4, 2, kAny},
                              {4, 4, 4, kAny},  {4, 4, 8, kAny}, {2, 4, 8, kAny}, {1, 4, 8, kAny}};
  static const Shape bwd_odd[] = {{32, 4, 1, kAny}, {16, 4, 1, kAny}, {8, 4, 1, kAny}, {8, 4, 2, kAny},
                                  {8, 4, 4, kAny},  {8, 4, 8, kAny},  {4, 4, 8, kAny}, {2, 4, 8, kAny}};
  const Shape* s = !forward ? (g->shifted ? bwd_odd : bwd) : !g->shifted ? fwd : fwd_odd;
  const int ns = forward ? 11 : 8;
  int best = 0;
  for (int k = 0; k < ns; ++k) {
    int LX = s[k].LX;
    if (LX <= spare) break;
    if (C > s[k].most) continue;
    while (LX > 1 + spare && LX / 2 >= words) LX /= 2;
    // fewer pixels to a tile while there are not two tiles for each SM
    while (LX > 4 && B * ((words + LX - 1) / LX) < 2 * kSMs) LX /= 2;
    const int cpc = (C + s[k].CL - 1) / s[k].CL, block = g->apart * s[k].NCH;  // channels of `apart` threads
    const int NL = (cpc + block - 1) / block * g->apart;
    if ((long long)LX * NL > kMaxThreads) continue;
    while (LX * NL < 32 && LX < 32) LX *= 2;  // a warp at least
    const int NT = (LX * NL + 31) / 32 * 32, threads = NT * (kMaxThreads / NT);
    if (threads <= best) continue;
    // the ring, and a Joiner's sums (of two kinds in the gradient)
    const size_t sums = forward ? 1 : 2, slots = (size_t)g->V * (LX + spare);
    const size_t ring = (size_t)NT * s[k].NCH * 16 * (forward ? 2 : 3);
    if (ring + 4 * sums * ((NT / LX) * (slots + 36) + slots * (1 + 2 * s[k].CL)) + 64 > kMaxSmem) continue;
    best = threads;
    g->LX = LX, g->NCH = s[k].NCH, g->CL = s[k].CL, g->cpc = cpc, g->NT = NT;
    if (best >= kMaxThreads * 3 / 4 || s[k].CL > 1) break;
  }
  if (!best) return false;
  g->TP = (g->LX - spare) * g->V;
  g->finish(B, C, P, max(1, kSMs * (kMaxThreads / g->NT) / g->CL));
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
  NormArgs a{x, residual, weight, h, y, q, scale, eps, 1.0f / (float)C, 0, 0, B, C, P};
  a.NG = groups(C, group, &a.G);
  if (!q) a.G = C, a.NG = 1;
  const size_t n = (size_t)B * C * P, e = elem_bytes(dtype);
  const Buffer in[] = {{x, n * e, "x"}, {residual, n * e, "residual"}, {weight, C * e, "weight"}};
  const Buffer out[] = {{h, n * e, "h"}, {y, n * e, "y"}, {q, n, "q"}, {scale, (size_t)B * a.NG * P * 4, "scale"}};
  const unsigned in_place[] = {3, 3, 0};
  if ((rc = check_buffers(in, in_place, 3, out, 4))) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
  rc = P == 1 ? norm_by_rows(a, dtype, st) : q ? norm_q_by_tiles(a, dtype, st) : norm_by_tiles(a, dtype, st);
  if (rc != DISCO_ERR_UNSUPPORTED) return rc;
  const long long tiles = (long long)B * ((P + 31) / 32);
  const int grid = (int)min(tiles, (long long)kSMs * 8);
#define CALL(T)                                                                     \
  if (P == 1) norm_any_kernel<T, true><<<grid, kGenWarps * 32, 0, st>>>(a, tiles);  \
  else norm_any_kernel<T, false><<<grid, kGenWarps * 32, 0, st>>>(a, tiles)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("norm_any_kernel");
}
