// disco_tokens.cu -- the 8-bit form of an activation's tokens (disco_quant_i8) and
// the gated activation (disco_glu), on activations [B, C, P]: checks, the choice
// of a kernel, and the general one.
//
//   y = act(x[:, :C]) x[:, C:]                    (disco_glu)
//   a = max(1e-30, max_c |v_c|), scale = a / 127, q_c = round(127 v_c / a)
//   for v = x (disco_quant_i8, and the checkpoint of disco_glu) and v = y (disco_glu)
//
// Tokens that a CTA holds in registers go by disco_tokens.cuh.  The general kernel
// below takes every other one and reads its inputs once for the largest magnitude
// and once more for the rounding.

#include "disco_tokens.cuh"

namespace disco {

DISCO_BOUNDS_READER(tokens_bounds)

namespace {

using namespace i8;

constexpr int kAnyThreads = 256;

// ROW: a block takes one token (P = 1), its threads the channels.  Else 32 pixels by 8 lanes of channels.
template <typename T, bool ROW, bool GLU>
__global__ void __launch_bounds__(kAnyThreads) tokens_any_kernel(const TokenArgs a, const long long tiles) {
  __shared__ float part[2][kAnyThreads];
  const int lx = ROW ? 0 : threadIdx.x & 31, j0 = ROW ? threadIdx.x : threadIdx.x >> 5, step = ROW ? kAnyThreads : kAnyThreads / 32;
  const long long per_sample = ROW ? 1 : (a.P + 31) / 32;
  const int NC = GLU ? 2 * a.C : a.C;
  const T* x = (const T*)a.x;
  for (long long t = blockIdx.x; t < tiles; t += gridDim.x) {
    const long long b = t / per_sample, p = (t - b * per_sample) * 32 * !ROW + lx;
    const bool live = p < a.P;
    const long long x0 = b * NC * a.P + p, y0 = b * a.C * a.P + p;
    auto value = [&](int c) { return gated<T, 1>({{to_f32(x[x0 + c * a.P])}}, {{to_f32(x[x0 + (c + a.C) * a.P])}}, a.act).v[0]; };
    // the largest of all threads of a token, NaN above all
    auto join = [&](float m, float* buf) {
      buf[threadIdx.x] = m;
      __syncthreads();
      uint32_t r = 0;
      if (ROW) {
        for (int k = 0; k < kAnyThreads; ++k) r = max(r, __float_as_uint(buf[k]));
      } else {
        for (int k = 0; k < kAnyThreads / 32; ++k) r = max(r, __float_as_uint(buf[lx + 32 * k]));
      }
      return __uint_as_float(r);
    };
    float mx = 0.0f, my = 0.0f;
    if (live) {
      if (a.xq)
        for (int c = j0; c < NC; c += step) mx = __uint_as_float(max32(__float_as_uint(mx), __float_as_uint(to_f32(x[x0 + c * a.P]))));
      if (GLU && (a.q || a.y))
        for (int c = j0; c < a.C; c += step) {
          const float v = value(c);
          my = max_abs(my, v);
          if (a.y) ((T*)a.y)[y0 + c * a.P] = from_f32<T>(v);
        }
    }
    if (a.xq) {
      const Quantizer z(join(mx, part[0]));
      if (live) {
        if (j0 == 0) a.xscale[b * a.P + p] = z.scale;
        for (int c = j0; c < NC; c += step) a.xq[x0 + c * a.P] = (int8_t)quantize<T>(to_f32(x[x0 + c * a.P]), z);
      }
    }
    if (GLU && a.q) {
      const Quantizer z(join(my, part[1]));
      if (live) {
        if (j0 == 0) a.scale[b * a.P + p] = z.scale;
        for (int c = j0; c < a.C; c += step) a.q[y0 + c * a.P] = (int8_t)quantize_y<T>(value(c), z);
      }
    }
    __syncthreads();
  }
}

template <typename T, bool GLU>
int any(const TokenArgs& a, cudaStream_t st) {
  const long long tiles = a.P == 1 ? a.B : a.B * ((a.P + 31) / 32);
  const int ctas = (int)min(tiles, (long long)kSMs * 8);
  if (a.P == 1) tokens_any_kernel<T, true, GLU><<<ctas, kAnyThreads, 0, st>>>(a, tiles);
  else tokens_any_kernel<T, false, GLU><<<ctas, kAnyThreads, 0, st>>>(a, tiles);
  return check_launch("tokens_any_kernel");
}

int tokens(const TokenArgs& a, bool glu, disco_dtype dtype, cudaStream_t st) {
  int rc = DISCO_ERR_UNSUPPORTED;
  if (a.P > 1) rc = a.P % (16 / elem_bytes(dtype)) == 0 ? tokens_grid(a, glu, dtype, st) : tokens_grid_odd(a, glu, dtype, st);
  if (rc == DISCO_ERR_UNSUPPORTED) rc = tokens_held(a, glu, dtype, st);
  if (rc != DISCO_ERR_UNSUPPORTED) return rc;
#define CALL(T) rc = glu ? any<T, true>(a, st) : any<T, false>(a, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

// ---- gradient of the gated activation at the checkpoint --------------------

struct GluBwdArgs {
  const void* dy;
  const int8_t* xq;
  const float* xscale;
  void* dx;
  int act, C;
  long long P, n;  // n = B C P elements of dy
};

// The gradients of a word's gates and values.
template <typename T, int V>
__device__ __forceinline__ void glu_bwd_word(const typename Word<V>::type& wg, const typename Word<V>::type& wv, const Raw<T, V>& wd, const float (&s)[V],
                                             int act, F<V>* dg, F<V>* dv) {
  uint32_t qg[(V + 3) / 4] = {}, qv[(V + 3) / 4] = {};
  memcpy(qg, &wg, V);
  memcpy(qv, &wv, V);
  const F<V> d = unpack<T, V>(wd);
#pragma unroll
  for (int e = 0; e < V; ++e) {
    const float g = from_byte(qg[e / 4] ^ 0x80808080u, e & 3) * s[e], v = from_byte(qv[e / 4] ^ 0x80808080u, e & 3) * s[e];
    float val;
    const float der = act_grad<T>(g, act, &val);
    dg->v[e] = d.v[e] * v * der;
    dv->v[e] = d.v[e] * val;
  }
}

// The word of V bytes at `at` of a tensor that ends within it.
template <int V>
__device__ __forceinline__ void memcpy_tail(void* w, const int8_t* x, long long at, long long total) {
  uint8_t v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = at + e < total ? (uint8_t)x[at + e] : 0;
  memcpy(w, v, V);
}

// Bound by HBM: [2,128,361x720] bf16 90 us, 5.9 TB/s; 16384 rows of 2048 45 us, 6.0 TB/s.
// Words of V neighbouring elements; a word is inside one channel's pixels (grids:
// V divides P) or one row's gates (rows: V divides C).  ROW: P = 1.
template <typename T, int V, bool ROW>
__global__ void __launch_bounds__(256) glu_bwd_kernel(const GluBwdArgs a) {
  using WQ = typename Word<V>::type;
  const long long i = (blockIdx.x * 256LL + threadIdx.x) * V;
  if (i >= a.n) return;
  const long long CP = a.C * a.P;
  const long long b = a.n <= 0xffffffffLL ? (long long)((uint32_t)i / (uint32_t)CP) : i / CP;
  const long long r = i - b * CP, g0 = 2 * b * CP + r;
  float s[V];
  const WQ wg = load_stream<WQ>(a.xq + g0), wv = load_stream<WQ>(a.xq + g0 + CP);
  const Raw<T, V> wd = load_stream<Raw<T, V>>((const T*)a.dy + i);
  if constexpr (ROW) {
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = a.xscale[b];
  } else {
    const long long p = r <= 0xffffffffLL && a.P <= 0xffffffffLL ? (long long)((uint32_t)r % (uint32_t)a.P) : r % a.P;
    if constexpr (V % 4 == 0) {
#pragma unroll
      for (int e = 0; e < V; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(a.xscale + b * a.P + p + e);
        s[e] = f.x, s[e + 1] = f.y, s[e + 2] = f.z, s[e + 3] = f.w;
      }
    } else {
      s[0] = a.xscale[b * a.P + p];
    }
  }
  F<V> dg, dv;
  glu_bwd_word<T, V>(wg, wv, wd, s, a.act, &dg, &dv);
  store_stream((T*)a.dx + g0, packed<T, V>(dg));
  store_stream((T*)a.dx + g0 + CP, packed<T, V>(dv));
}

// Grids where V does not divide P: a warp takes 32 V pixels of a channel; aligned words are
// shifted to pixels on the way in and back on the way out (disco_tokens.cuh).
// [2,128,361x719] bf16: 176 us; one pixel to a thread 304.
template <typename T>
__global__ void __launch_bounds__(256) glu_bwd_odd_kernel(const GluBwdArgs a, const long long per_row, const long long units) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES;
  using WQ = typename Word<V>::type;
  const int lane = threadIdx.x & 31;
  const long long unit = blockIdx.x * 8LL + threadIdx.x / 32;
  if (unit >= units) return;  // the whole warp
  const long long row = units <= 0xffffffffLL ? (long long)((uint32_t)unit / (uint32_t)per_row) : unit / per_row;
  const long long b = row / a.C, pos = (unit - row * per_row) * (32 * V), half = a.C * a.P;
  const int N = (int)min(32LL * V, a.P - pos), nv = min(V, N - lane * V);
  const long long y0 = row * a.P + pos, g0 = y0 + b * half, p = pos + lane * V;  // dy's first element, the gate's
  WQ wg = {}, wv = {};
  uint4 wd = make_uint4(0, 0, 0, 0);
  float s[V] = {};
  if (nv > 0) {
    auto q8 = [&](long long k) {  // V integers from element k on
      const int m = (int)k & (V - 1);
      const long long at = k - m;
      WQ lo = {}, hi = {};
      if (at + V <= 2 * a.n) lo = load_stream<WQ>(a.xq + at);
      else memcpy_tail<V>(&lo, a.xq, at, 2 * a.n);
      if (m + nv > V) {
        if (at + 2 * V <= 2 * a.n) hi = load_stream<WQ>(a.xq + at + V);
        else memcpy_tail<V>(&hi, a.xq, at + V, 2 * a.n);
      }
      uint32_t u[V / 2 + 1] = {};
      memcpy(u, &lo, V);
      memcpy(u + V / 4, &hi, V);
      if (V == 8 && (m & 4)) u[0] = u[1], u[1] = u[2], u[2] = u[3];
      uint32_t o[V / 4];
#pragma unroll
      for (int i = 0; i < V / 4; ++i) o[i] = __funnelshift_r(u[i], u[i + 1], 8 * (m & 3));
      WQ w;
      memcpy(&w, o, V);
      return w;
    };
    wg = q8(g0 + lane * V), wv = q8(g0 + half + lane * V);
    wd = load_px<T, V>((const T*)a.dy, y0 + lane * V, nv, a.n);
#pragma unroll
    for (int e = 0; e < V; ++e) s[e] = e < nv ? a.xscale[b * a.P + p + e] : 0.0f;
  }
  F<V> dg, dv;
  glu_bwd_word<T, V>(wg, wv, wd, s, a.act, &dg, &dv);
  store_px<V>(a.dx, g0, packed<T, V>(dg), lane, 32, N, true);
  store_px<V>(a.dx, g0 + half, packed<T, V>(dv), lane, 32, N, true);
}

template <typename T, int V>
int glu_bwd(const GluBwdArgs& a, cudaStream_t st) {
  const long long grid = (a.n / V + 255) / 256;
  if (grid > 0x7fffffffLL) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^31 - 1 blocks of %d elements", 256 * V);
  if (a.P == 1) glu_bwd_kernel<T, V, true><<<(unsigned)grid, 256, 0, st>>>(a);
  else glu_bwd_kernel<T, V, false><<<(unsigned)grid, 256, 0, st>>>(a);
  return check_launch("glu_bwd_kernel");
}

template <typename T>
int glu_bwd_odd(const GluBwdArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  const long long per_row = (a.P + 32 * V - 1) / (32 * V), units = a.n / a.P * per_row, grid = (units + 7) / 8;
  if (grid > 0x7fffffffLL) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^31 - 1 blocks of 8 times %d pixels", 32 * V);
  glu_bwd_odd_kernel<T><<<(unsigned)grid, 256, 0, st>>>(a, per_row, units);
  return check_launch("glu_bwd_odd_kernel");
}

int check_act(int32_t kind) {
  if (kind != DISCO_SILU && kind != DISCO_GELU) return fail(DISCO_ERR_UNSUPPORTED, "activation");
  return DISCO_OK;
}

}  // namespace
}  // namespace disco

using namespace disco;
using namespace disco::i8;

extern "C" int disco_quant_i8(const void* x, void* q, float* scale, int32_t B, int32_t C, int64_t P, disco_dtype dtype,
                              void* stream) {
  disco::NvtxScope nvtx_scope("disco_quant_i8");
  int rc;
  if ((rc = check_shape(B, C, P, dtype))) return rc;
  if (!x || !q || !scale) return fail(DISCO_ERR_INVALID_ARG, "x, q or scale is null");
  if ((rc = check_device())) return rc;
  const size_t n = (size_t)B * C * P;
  const Buffer in[] = {{x, n * elem_bytes(dtype), "x"}};
  const Buffer out[] = {{q, n, "q"}, {scale, (size_t)B * P * 4, "scale"}};
  const unsigned in_place[] = {0};
  if ((rc = check_buffers(in, in_place, 1, out, 2))) return rc;
  const TokenArgs a{x, nullptr, nullptr, nullptr, (int8_t*)q, scale, DISCO_SILU, B, C, P};
  return tokens(a, false, dtype, (cudaStream_t)stream);
}

extern "C" int disco_glu(const void* x, void* y, void* q, float* scale, void* xq, float* xscale, disco_activation act,
                         int32_t B, int32_t C, int64_t P, disco_dtype dtype, void* stream) {
  disco::NvtxScope nvtx_scope("disco_glu");
  int rc;
  if ((rc = check_shape(B, C, P, dtype)) || (rc = check_act(act))) return rc;
  if (C > 1 << 29) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^29 channels");
  if (!x) return fail(DISCO_ERR_INVALID_ARG, "x is null");
  if (!y && !q) return fail(DISCO_ERR_INVALID_ARG, "neither y nor q is given");
  if (!q != !scale) return fail(DISCO_ERR_INVALID_ARG, "q and scale come together");
  if (!xq != !xscale) return fail(DISCO_ERR_INVALID_ARG, "xq and xscale come together");
  if ((rc = check_device())) return rc;
  const size_t n = (size_t)B * C * P, e = elem_bytes(dtype), t = (size_t)B * P * 4;
  const Buffer in[] = {{x, 2 * n * e, "x"}};
  const Buffer out[] = {{y, n * e, "y"}, {q, n, "q"}, {scale, t, "scale"}, {xq, 2 * n, "xq"}, {xscale, t, "xscale"}};
  const unsigned in_place[] = {0};
  if ((rc = check_buffers(in, in_place, 1, out, 5))) return rc;
  const TokenArgs a{x, y, (int8_t*)q, scale, (int8_t*)xq, xscale, act, B, C, P};
  return tokens(a, true, dtype, (cudaStream_t)stream);
}

extern "C" int disco_glu_bwd(const void* dy, const void* xq, const float* xscale, void* dx, disco_activation act, int32_t B,
                             int32_t C, int64_t P, disco_dtype dtype, void* stream) {
  disco::NvtxScope nvtx_scope("disco_glu_bwd");
  int rc;
  if ((rc = check_shape(B, C, P, dtype)) || (rc = check_act(act))) return rc;
  if (C > 1 << 29) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^29 channels");
  if (!dy || !xq || !xscale || !dx) return fail(DISCO_ERR_INVALID_ARG, "dy, xq, xscale or dx is null");
  if ((rc = check_device())) return rc;
  const size_t n = (size_t)B * C * P, e = elem_bytes(dtype);
  const Buffer in[] = {{dy, n * e, "dy"}, {xq, 2 * n, "xq"}, {xscale, (size_t)B * P * 4, "xscale"}};
  const Buffer out[] = {{dx, 2 * n * e, "dx"}};
  const unsigned in_place[] = {0, 0, 0};
  if ((rc = check_buffers(in, in_place, 3, out, 1))) return rc;
  const GluBwdArgs a{dy, (const int8_t*)xq, xscale, dx, act, C, P, (long long)n};
#define CALL(T)                                                                          \
  if ((P == 1 ? C : P) % (16 / (int)sizeof(T)) == 0) rc = glu_bwd<T, 16 / (int)sizeof(T)>(a, (cudaStream_t)stream); \
  else if (P >= 64) rc = glu_bwd_odd<T>(a, (cudaStream_t)stream); /* fewer pixels leave a warp idle */ \
  else rc = glu_bwd<T, 1>(a, (cudaStream_t)stream)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}
