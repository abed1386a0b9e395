// disco_grad.cu -- the Euclidean norm over all gradients of a model and their
// scaling to a largest norm (disco_grad_norm, disco_grad_clip).
//
// The list of gradients travels in the kernels' parameters, so a call depends
// on no device table and no earlier copy.  Work is cut into chunks that do not
// cross tensors, dealt to the warps of persistent CTAs in turn: a warp's chunk
// may be a bias of a few elements without idling a CTA.
//
// Sums of squares are kept at three scales, sum g^2, sum (g 2^-80)^2 and
// sum (g 2^90)^2: where the first is infinite the second holds the answer,
// where it is below 2^-60 (its terms near the smallest fp32) the third.  All
// in fp32 (all terms are positive, threads and CTAs join pairwise; the few
// fp64 units of this GPU took longer than the loads): a CTA leaves one row of
// partial sums, and every CTA of the scaling kernel adds those rows up for
// itself: two launches, no atomics, one order of summation.  A short list runs
// in one launch of one cluster, whose CTAs exchange their rows through
// distributed shared memory.
//
// Bound by HBM for long lists (every gradient is read twice where they do not fit
// on the chip, and written once), by launches for short ones.  Measured (GB300):
// 48 gradients of [512,512,9] bf16 into fp32, 679 MB and 226 MB read again: norm 37
// us (6.1 TB/s), both 144.5 us a call, into bf16 119, in place 101; 8 of [64,64,3]
// 7.2 to 8.4 us (by host); 240 ragged ones of two types (2.5 million elements, outs
// packed back to back) 12.4 us; 32 thousand elements in the one cluster 7.2 us, in two launches 8.9,
// 262 thousand 16.4 and 9.0, hence kSmall.

#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "disco_bounds.cuh"
#include "disco_internal.cuh"

namespace disco {

DISCO_BOUNDS_READER(grad_bounds)

namespace {

constexpr int kThreads = 256;
constexpr int kSMs = 152;
constexpr int kNormPerSM = 4, kClipPerSM = 2;  // resident CTAs of the large kernels
constexpr int kNormGrid = kSMs * kNormPerSM;   // CTAs of a norm launch at most = rows of its partial sums
constexpr int kClipGrid = kSMs * kClipPerSM;
constexpr int kNormUnroll = 8, kClipUnroll = 4;  // 16-byte loads a lane has in flight
// Longest chunks, in elements.  Scaling writes as it reads: with one round of a
// warp's 16-bit loads to a chunk the warps of a CTA stay side by side in memory
// (1024: 113 us for 113 million bf16 elements into fp32; 2048: 116; 4 CTAs to an
// SM: 123).  The norm only reads (8192: 45 us, 1024: 54).
constexpr int kNormChunk = 8192, kClipChunk = 1024;
constexpr int kCluster = 16;                     // CTAs of the small kernel

struct Entry {
  const void* g;
  void* o;
  long long n;
  int chunk0;        // first chunk of the tensor
  short dt, odt;
};
// The gradients of one launch; kernel parameters end at 32,764 bytes, and a
// launch costs more the longer they are.
template <int N>
struct Table {
  Entry e[N];
  long long chunk;   // elements of a chunk
  int chunks, count;
};
constexpr int kShort = 64, kMiddle = 256, kLong = 1000;
static_assert(sizeof(Table<kLong>) + 64 <= 32764, "kernel parameters");

// the tensor that chunk c belongs to; `at`: the last answer, often this one too
template <int N>
__device__ __forceinline__ const Entry& find(const Table<N>& t, int c, int& at) {
  if (c < t.e[at].chunk0 || (at + 1 < t.count && c >= t.e[at + 1].chunk0)) {
    int lo = 0, hi = t.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (t.e[mid].chunk0 <= c) lo = mid;
      else hi = mid - 1;
    }
    at = lo;
  }
  return t.e[at];
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 x, y, z, w;\n"
      "mov.b64 x, {%2, %3}; mov.b64 y, {%4, %5}; mov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 w, x, y, z;\n"
      "mov.b64 {%0, %1}, w;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float s) {
  float2 r;
  asm("{.reg .b64 x, y, w;\n"
      "mov.b64 x, {%2, %3}; mov.b64 y, {%4, %4};\n"
      "mul.rn.f32x2 w, x, y;\n"
      "mov.b64 {%0, %1}, w;}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(s));
  return r;
}

// The three sums of a thread, two terms at a time.
struct Sums {
  float2 a = {0.0f, 0.0f}, b = {0.0f, 0.0f}, c = {0.0f, 0.0f};
  template <typename T>
  __device__ __forceinline__ void add(float2 v) {
    a = fma2(v, v, a);
    if constexpr (!__is_same(T, __half)) {
      const float2 u = mul2(v, 0x1p-80f), w = mul2(v, 0x1p90f);
      b = fma2(u, u, b);
      c = fma2(w, w, c);
    }
  }
  // fp16 squares lie within fp32's range: their sum stands in the first alone,
  // and an infinity or NaN in all
  __device__ __forceinline__ void add_f16(const Sums& s) {
    const float z = s.a.x + s.a.y;
    a.x += z;
    if (!isfinite(z)) b.x = c.x = z;
  }
};

template <typename T>
__device__ __forceinline__ void sum_word(Sums& s, const uint4& w) {
  T t[16 / sizeof(T)];
  memcpy(t, &w, 16);
#pragma unroll
  for (int e = 0; e < (int)(16 / sizeof(T)); e += 2) s.add<T>(make_float2(to_f32(t[e]), to_f32(t[e + 1])));
}

// elements [i0, i1) of a tensor, by one warp; i0 is a multiple of 16
template <typename T>
__device__ __forceinline__ void sum_elements(Sums& s, const T* g, long long i0, long long i1) {
  constexpr int V = 16 / sizeof(T);
  const int lane = threadIdx.x & 31;
  g += i0;
  const int n = (int)(i1 - i0);
  int i = 0;
  if (((uintptr_t)g & 15) == 0) {
    const uint4* p = (const uint4*)g;
    const int words = n / V;
    int k = lane;
    for (; k + (kNormUnroll - 1) * 32 < words; k += kNormUnroll * 32) {
      uint4 w[kNormUnroll];
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) w[u] = p[k + u * 32];
#pragma unroll
      for (int u = 0; u < kNormUnroll; ++u) sum_word<T>(s, w[u]);
    }
    for (; k < words; k += 32) sum_word<T>(s, p[k]);
    i = words * V;
  }
  // the rest, and tensors off a 16-byte boundary, by elements
  for (i += lane; i < n; i += 8 * 32) {
    T t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) t[u] = i + u * 32 < n ? g[i + u * 32] : from_f32<T>(0.0f);
#pragma unroll
    for (int u = 0; u < 8; u += 2) s.add<T>(make_float2(to_f32(t[u]), to_f32(t[u + 1])));
  }
}

struct Row {
  float v[3];
};
// The sums over the CTA's threads, in one order, to all of them.
__device__ __forceinline__ Row cta_sum(Row r, Row* buf) {
#pragma unroll
  for (int m = 16; m; m >>= 1)
#pragma unroll
    for (int n = 0; n < 3; ++n) r.v[n] += __shfl_xor_sync(0xffffffffu, r.v[n], m);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x / 32] = r;
  __syncthreads();
  r = buf[0];
#pragma unroll
  for (int k = 1; k < kThreads / 32; ++k)
#pragma unroll
    for (int n = 0; n < 3; ++n) r.v[n] += buf[k].v[n];
  return r;
}
__device__ __forceinline__ Row row_of(const Sums& s) { return Row{{s.a.x + s.a.y, s.b.x + s.b.y, s.c.x + s.c.y}}; }
// The scaled norm.  Where the root lies outside fp32's range, or might be rounded among
// its subnormals, powers of two are joined last: the product may lie inside it.
__device__ __forceinline__ float norm_of(const Row& r, float grad_scale) {
  float v = r.v[0];
  if (!(isinf(v) || v < 0x1p-60f)) return sqrtf(v) * grad_scale;
  int e;
  const float m = frexpf(grad_scale, &e);
  if (isinf(v)) v = r.v[1], e += 80;
  else v = r.v[2], e -= 90;
  return scalbnf(sqrtf(v) * m, e);
}

// A CTA's warps take neighbouring chunks.
constexpr int kWarps = kThreads / 32;
__device__ __forceinline__ int first_chunk() { return blockIdx.x * kWarps + threadIdx.x / 32; }

// chunk k's squares
template <int N>
__device__ __forceinline__ void sum_chunk(Sums& s, const Table<N>& t, int k, int& at) {
  const Entry& e = find(t, k, at);
  const long long i0 = (k - e.chunk0) * t.chunk, i1 = min(e.n, i0 + t.chunk);
  if (e.dt == DISCO_F32) sum_elements(s, (const float*)e.g, i0, i1);
  else if (e.dt == DISCO_BF16) sum_elements(s, (const __nv_bfloat16*)e.g, i0, i1);
  else {
    Sums h;
    sum_elements(h, (const __half*)e.g, i0, i1);
    s.add_f16(h);
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kNormPerSM) grad_norm_kernel(const __grid_constant__ Table<N> t, Row* part) {
  __shared__ Row buf[kThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;");
  Sums s;
  int at = 0;
  for (int k = first_chunk(); k < t.chunks; k += gridDim.x * kWarps) sum_chunk(s, t, k, at);
  const Row r = cta_sum(row_of(s), buf);
  if (threadIdx.x == 0) part[blockIdx.x] = r;
}

// All rows of partial sums, to every thread of the CTA.
__device__ __forceinline__ Row sum_rows(const Row* part, int parts, Row* buf) {
  Row r{{0.0f, 0.0f, 0.0f}};
  for (int i = threadIdx.x; i < parts; i += kThreads)
#pragma unroll
    for (int n = 0; n < 3; ++n) r.v[n] += part[i].v[n];
  return cta_sum(r, buf);
}

__global__ void __launch_bounds__(kThreads) grad_norm_finish_kernel(const Row* part, int parts, float grad_scale, float* norm) {
  __shared__ Row buf[kThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float v = norm_of(sum_rows(part, parts, buf), grad_scale);
  if (threadIdx.x == 0) *norm = v;
}

template <int BYTES> struct Word;
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };

// Factor a b of the clipped gradients, out = (g a) b.  a = 1 but for a product that
// nears fp32's subnormals (gradients 2^100 times past max_norm): it is split evenly
// there, so that neither factor is rounded among them.
struct Factor {
  float a, b;
};
__device__ __forceinline__ Factor factor(float norm, float grad_scale, float max_norm) {
  if (norm <= max_norm) return {1.0f, grad_scale};
  const float q = max_norm / norm, f = grad_scale * q;
  if ((q >= 0x1p-100f && f >= 0x1p-100f) || !(norm < INFINITY)) return {1.0f, f};  // or 0, or NaN
  int es, em, en;
  const float m = frexpf(grad_scale, &es) * (frexpf(max_norm, &em) / frexpf(norm, &en));
  const int e = es + em - en, half = e < -100 ? e / 2 : 0;
  return {scalbnf(1.0f, half), scalbnf(m, e - half)};
}

// out = g f of elements [i0, i1), by one warp.  A lane takes V elements, 16 bytes of
// the wider side, so that both the loads and the stores of a warp lie side by side.
template <typename T, typename O>
__device__ __forceinline__ void clip_elements(const T* g, O* o, long long i0, long long i1, Factor f) {
  constexpr int V = 16 / (sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O));
  constexpr int U = sizeof(T) < sizeof(O) ? 2 * kClipUnroll : kClipUnroll;  // loads in flight, of 8 or 16 bytes
  using WT = typename Word<V * (int)sizeof(T)>::type;
  using WO = typename Word<V * (int)sizeof(O)>::type;
  const int lane = threadIdx.x & 31;
  g += i0;
  o += i0;
  const int n = (int)(i1 - i0);
  int i = 0;
  if ((((uintptr_t)g | (uintptr_t)o) & 15) == 0) {
    const WT* p = (const WT*)g;
    const int words = n / V;
    auto put = [&](const WT& w, int k) {
      T t[V];
      O r[V];
      WO z;
      memcpy(t, &w, sizeof(w));
#pragma unroll
      for (int e = 0; e < V; ++e) r[e] = from_f32<O>(to_f32(t[e]) * f.a * f.b);
      memcpy(&z, r, sizeof(z));
      __stcs((WO*)o + k, z);
    };
    int k = lane;
    for (; k + (U - 1) * 32 < words; k += U * 32) {
      WT w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) w[u] = __ldcs(p + k + u * 32);
#pragma unroll
      for (int u = 0; u < U; ++u) put(w[u], k + u * 32);
    }
    for (; k < words; k += 32) put(__ldcs(p + k), k);
    i = words * V;
  }
  for (i += lane; i < n; i += 8 * 32) {
    T t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u * 32 < n) t[u] = g[i + u * 32];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u * 32 < n) o[i + u * 32] = from_f32<O>(to_f32(t[u]) * f.a * f.b);
  }
}

template <typename T>
__device__ __forceinline__ void clip_entry(const Entry& e, long long i0, long long i1, Factor f) {
  if (e.odt == DISCO_F32) clip_elements((const T*)e.g, (float*)e.o, i0, i1, f);
  else if (e.odt == DISCO_BF16) clip_elements((const T*)e.g, (__nv_bfloat16*)e.o, i0, i1, f);
  else clip_elements((const T*)e.g, (__half*)e.o, i0, i1, f);
}

template <int N>
__device__ __forceinline__ void clip_chunk(const Table<N>& t, int k, int& at, Factor f) {
  const Entry& e = find(t, k, at);
  if (e.o == e.g && f.b == 1.0f) return;  // then a is 1 too
  const long long i0 = (k - e.chunk0) * t.chunk, i1 = min(e.n, i0 + t.chunk);
  if (e.dt == DISCO_F32) clip_entry<float>(e, i0, i1, f);
  else if (e.dt == DISCO_BF16) clip_entry<__nv_bfloat16>(e, i0, i1, f);
  else clip_entry<__half>(e, i0, i1, f);
}

// part: the rows of partial sums of this call's norm (the norm is written to
// *norm by CTA 0), or null: the norm is read from *norm.
template <int N>
__global__ void __launch_bounds__(kThreads, kClipPerSM)
    grad_clip_kernel(const __grid_constant__ Table<N> t, const Row* part, int parts, float grad_scale, float max_norm, float* norm) {
  __shared__ Row buf[kThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float n;
  if (part) {
    n = norm_of(sum_rows(part, parts, buf), grad_scale);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  } else {
    n = *norm;
  }
  const Factor f = factor(n, grad_scale, max_norm);
  int at = 0;
  // last chunks first: the norm's pass read them last, they may still be in L2
  for (int k = t.chunks - 1 - first_chunk(); k >= 0; k -= gridDim.x * kWarps) clip_chunk(t, k, at, f);
}

// A short list in one launch: the CTAs of one cluster take its chunks in turn,
// push their rows of sums to one another, and scale the chunks they summed.
template <int N>
__global__ void __launch_bounds__(kThreads)
    grad_small_kernel(const __grid_constant__ Table<N> t, float grad_scale, float max_norm, bool clip, float* norm) {
  __shared__ Row buf[kThreads / 32], box[kCluster];
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  Sums s;
  int at = 0;
  for (int k = first_chunk(); k < t.chunks; k += kCluster * kWarps) sum_chunk(s, t, k, at);
  Row r = cta_sum(row_of(s), buf);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA runs: its memory may be written
  if (threadIdx.x < kCluster) {
    uint32_t to;
    asm("mapa.shared::cluster.u32 %0, %1, %2;"
        : "=r"(to)
        : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(&box[blockIdx.x]))), "r"(threadIdx.x));
#pragma unroll
    for (int n = 0; n < 3; ++n) asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + 4 * n), "f"(r.v[n]) : "memory");
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  r = box[0];
#pragma unroll
  for (int k = 1; k < kCluster; ++k)
#pragma unroll
    for (int n = 0; n < 3; ++n) r.v[n] += box[k].v[n];
  const float n = norm_of(r, grad_scale);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
  if (!clip) return;
  const Factor f = factor(n, grad_scale, max_norm);
  for (int k = first_chunk(); k < t.chunks; k += kCluster * kWarps) clip_chunk(t, k, at, f);
}

// Elements of a chunk (a warp's): two for each warp of the norm's grid where
// there is enough work, from 256 (one 16-byte load of 16-bit elements for each
// lane) to `most`, and more where there would be more than 2^27 chunks.
long long chunk_of(const disco_grads* g, int most) {
  long long c = 256;
  while (c < most && g->numel / c > 2 * kNormGrid * kWarps) c *= 2;
  while (g->numel / c > (1 << 27)) c *= 2;
  return c;
}

// Fills `t` from tensors[*next ...]; false when none with elements is left.
template <int N>
bool fill(const disco_grads* g, int* next, int most, Table<N>* t) {
  t->count = 0;
  t->chunks = 0;
  t->chunk = chunk_of(g, most);
  for (; *next < g->count && t->count < N; ++*next) {
    const disco_grad_tensor& s = g->tensors[*next];
    if (s.n < 1) continue;
    t->e[t->count++] = Entry{s.grad, s.out, s.n, t->chunks, (short)s.dtype, (short)s.out_dtype};
    t->chunks += (int)((s.n + t->chunk - 1) / t->chunk);
  }
  return t->count > 0;
}

// A launch that may begin while the kernel before it on the stream ends; the
// kernel waits (griddepcontrol.wait) before it reads what that one wrote.
template <typename K, typename... A>
cudaError_t launch_after(K kernel, int grid, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int launch_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DISCO_OK;
  (void)cudaGetLastError();
  return fail(DISCO_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
}

// at most: norm launches of a list
int launches(const disco_grads* g) { return g->count / kLong + 1; }

int elem_bytes(int dt) { return dt == DISCO_F32 ? 4 : 2; }

struct Span {
  const char *lo, *hi;
  int32_t i;
  bool out;
};
int by_lo(const void* a, const void* b) {
  const Span *u = (const Span*)a, *v = (const Span*)b;
  return u->lo < v->lo ? -1 : u->lo > v->lo;
}

// No out may overlap another out or a gradient other than its own, and its
// own only from the same address with the same type.
int check_overlaps(const disco_grad_tensor* t, int32_t count) {
  Span* s = (Span*)malloc(sizeof(Span) * 2 * (size_t)count);
  if (!s) return fail(DISCO_ERR_INVALID_ARG, "out of host memory for %d gradients", count);
  int32_t m = 0;
  for (int32_t i = 0; i < count; ++i) {
    if (t[i].n < 1) continue;
    const char *g = (const char*)t[i].grad, *o = (const char*)t[i].out;
    if (!o || o != g) s[m++] = Span{g, g + t[i].n * elem_bytes(t[i].dtype), i, false};
    if (o) s[m++] = Span{o, o + t[i].n * elem_bytes(t[i].out_dtype), i, true};
  }
  qsort(s, m, sizeof(Span), by_lo);
  int rc = DISCO_OK;
  // furthest ends seen so far of any span and of the outs
  const char *end = nullptr, *out_end = nullptr;
  int32_t end_i = 0, out_i = 0;
  for (int32_t k = 0; k < m && !rc; ++k) {
    if (s[k].out ? s[k].lo < end : s[k].lo < out_end)
      rc = fail(DISCO_ERR_INVALID_ARG, "out of gradient %d overlaps a buffer of gradient %d", s[k].out ? s[k].i : out_i,
                s[k].out ? end_i : s[k].i);
    if (s[k].hi > end) end = s[k].hi, end_i = s[k].i;
    if (s[k].out && s[k].hi > out_end) out_end = s[k].hi, out_i = s[k].i;
  }
  free(s);
  return rc;
}

int check_grads(const disco_grads* g, float grad_scale) {
  if (!g) return fail(DISCO_ERR_INVALID_ARG, "grads is null");
  if (g->count < 0 || (g->count > 0 && !g->tensors)) return fail(DISCO_ERR_INVALID_ARG, "grads is not planned (call disco_grad_plan)");
  if (!(grad_scale > 0.0f) || isinf(grad_scale)) return fail(DISCO_ERR_INVALID_ARG, "grad_scale must be positive and finite");
  int rc = check_device(), dev = 0;
  if (rc) return rc;
  if (cudaGetDevice(&dev) != cudaSuccess || (g->numel > 0 && dev != g->device))
    return fail(DISCO_ERR_INVALID_ARG, "the gradients live on device %d, the current device is %d", g->device, dev);
  return DISCO_OK;
}

int check_scalar(const float* p, const char* name) {
  int rc = check_dev_ptr(p, name);
  if (rc) return rc;
  if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(DISCO_ERR_ALIGNMENT, "%s must be 4-byte aligned", name);
  return DISCO_OK;
}

int check_max_norm(const disco_grads* g, float max_norm) {
  if (!(max_norm >= 0.0f)) return fail(DISCO_ERR_INVALID_ARG, "max_norm must be >= 0");
  if (!g->has_out) return fail(DISCO_ERR_INVALID_ARG, "a gradient has no out");
  return DISCO_OK;
}

bool overlap(const void* p, size_t n, const void* q, size_t m) { return (uintptr_t)p < (uintptr_t)q + m && (uintptr_t)q < (uintptr_t)p + n; }

// No kernel may read or write the gradients (`grads`) and outs (`outs`) where another
// of the call writes the norm or partial sums (ws, null: none), nor these each other.
int check_apart(const disco_grads* g, bool grads, bool outs, const float* norm, const void* ws, size_t ws_bytes) {
  if (ws && overlap(norm, 4, ws, ws_bytes)) return fail(DISCO_ERR_INVALID_ARG, "norm overlaps the workspace");
  for (int32_t i = 0; i < g->count; ++i) {
    const disco_grad_tensor& t = g->tensors[i];
    if (t.n < 1) continue;
    for (int o = 0; o < 2; ++o) {
      if (!(o ? outs && t.out : grads)) continue;
      const void* p = o ? t.out : t.grad;
      const size_t bytes = (size_t)t.n * elem_bytes(o ? t.out_dtype : t.dtype);
      const char* what = overlap(norm, 4, p, bytes) ? "norm" : ws && overlap(ws, ws_bytes, p, bytes) ? "the workspace" : nullptr;
      if (what) return fail(DISCO_ERR_INVALID_ARG, "%s overlaps %sgradient %d", what, o ? "the out of " : "", i);
    }
  }
  return DISCO_OK;
}

// Elements of a list that one cluster takes.
constexpr long long kSmall = 1 << 16;

template <int N>
int run_small(const disco_grads* g, float grad_scale, float max_norm, bool clip, float* norm, cudaStream_t st) {
  Table<N> t;
  int next = 0;
  fill(g, &next, kClipChunk, &t);
  cudaError_t e = cudaFuncSetAttribute((const void*)grad_small_kernel<N>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, grad_small_kernel<N>, t, grad_scale, max_norm, clip, norm);
  }
  return launch_status(e, "grad_small_kernel");
}

// Partial sums of all gradients; *parts: rows.
template <int N>
int norm_parts(const disco_grads* g, Row* part, int* parts, cudaStream_t st) {
  Table<N> t;
  int next = 0;
  *parts = 0;
  while (fill(g, &next, kNormChunk, &t)) {
    const int ctas = (t.chunks + kWarps - 1) / kWarps, grid = ctas < kNormGrid ? ctas : kNormGrid;
    grad_norm_kernel<N><<<grid, kThreads, 0, st>>>(t, part + *parts);
    const int rc = launch_status(cudaGetLastError(), "grad_norm_kernel");
    if (rc) return rc;
    *parts += grid;
  }
  return DISCO_OK;
}

template <int N>
int clip_all(const disco_grads* g, const Row* part, int parts, float grad_scale, float max_norm, float* norm, cudaStream_t st) {
  Table<N> t;
  int next = 0;
  while (fill(g, &next, kClipChunk, &t)) {
    const int ctas = (t.chunks + kWarps - 1) / kWarps, grid = ctas < kClipGrid ? ctas : kClipGrid;
    const int rc = launch_status(launch_after(grad_clip_kernel<N>, grid, st, t, part, parts, grad_scale, max_norm, norm),
                                 "grad_clip_kernel");
    if (rc) return rc;
    part = nullptr;  // a further launch reads the norm
  }
  return DISCO_OK;
}

int finish_norm(const Row* part, int parts, float grad_scale, float* norm, cudaStream_t st) {
  return launch_status(launch_after(grad_norm_finish_kernel, 1, st, part, parts, grad_scale, norm), "grad_norm_finish_kernel");
}

// The norm, and with `clip` the scaled gradients, by tables of N.
template <int N>
int run(const disco_grads* g, float grad_scale, float max_norm, bool clip, float* norm, void* ws, cudaStream_t st) {
  // a list without elements, of any length, is a short one: its norm is written too
  if (g->numel == 0 || (g->count <= N && g->numel <= kSmall)) return run_small<N>(g, grad_scale, max_norm, clip, norm, st);
  Row* part = (Row*)ws;
  int parts, rc = norm_parts<N>(g, part, &parts, st);
  if (rc) return rc;
  return clip ? clip_all<N>(g, part, parts, grad_scale, max_norm, norm, st) : finish_norm(part, parts, grad_scale, norm, st);
}

#define DISCO_BY_COUNT(count, CALL)            \
  ((count) <= kShort    ? CALL(kShort)         \
   : (count) <= kMiddle ? CALL(kMiddle)        \
                        : CALL(kLong))

int run(const disco_grads* g, float grad_scale, float max_norm, bool clip, float* norm, void* ws, cudaStream_t st) {
#define CALL(N) run<N>(g, grad_scale, max_norm, clip, norm, ws, st)
  return DISCO_BY_COUNT(g->count, CALL);
#undef CALL
}

int check_workspace(const disco_grads* g, void* ws, size_t bytes) {
  const size_t need = disco_grad_workspace_bytes(g);
  if (!ws || bytes < need) return fail(DISCO_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned16(ws)) return fail(DISCO_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
  return check_dev_ptr(ws, "workspace");
}

}  // namespace
}  // namespace disco

using namespace disco;

extern "C" int disco_grad_plan(const disco_grad_tensor* tensors, int32_t count, disco_grads* grads) {
  disco::NvtxScope nvtx_scope("disco_grad_plan");
  if (!grads) return fail(DISCO_ERR_INVALID_ARG, "grads is null");
  *grads = disco_grads{};
  if (count < 0 || (count > 0 && !tensors)) return fail(DISCO_ERR_INVALID_ARG, "no tensors");
  int rc, dev = 0;
  disco_grads g{tensors, count, 1, 0, 0, 0};
  for (int32_t i = 0; i < count; ++i) {
    const disco_grad_tensor& t = tensors[i];
    if (t.n < 0) return fail(DISCO_ERR_INVALID_ARG, "gradient %d has %lld elements", i, (long long)t.n);
    if (t.n > (int64_t)1 << 50 || g.numel > (int64_t)1 << 50) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^50 elements");
    if (t.n == 0) continue;
    g.numel += t.n;
    if (t.dtype < DISCO_F32 || t.dtype > DISCO_F16 || (t.out && (t.out_dtype < DISCO_F32 || t.out_dtype > DISCO_F16)))
      return fail(DISCO_ERR_UNSUPPORTED, "dtype of gradient %d", i);
    if (!t.grad) return fail(DISCO_ERR_INVALID_ARG, "gradient %d is null", i);
    if (reinterpret_cast<uintptr_t>(t.grad) % elem_bytes(t.dtype) ||
        (t.out && reinterpret_cast<uintptr_t>(t.out) % elem_bytes(t.out_dtype)))
      return fail(DISCO_ERR_ALIGNMENT, "gradient %d or its out is not aligned to its element", i);
    if (t.out == t.grad && t.out_dtype != t.dtype)
      return fail(DISCO_ERR_INVALID_ARG, "out of gradient %d is in place with another dtype", i);
    if (!t.out) g.has_out = 0;
    else if (t.out == t.grad) g.in_place = 1;
  }
  if (g.numel > 0) {
    if ((rc = check_device()) || (rc = check_overlaps(tensors, count))) return rc;
    if (cudaGetDevice(&dev) != cudaSuccess) return fail(DISCO_ERR_CUDA, "cudaGetDevice failed");
    g.device = dev;
    char name[48];
    for (int32_t i = 0; i < count; ++i) {
      if (tensors[i].n == 0) continue;
      snprintf(name, sizeof name, "gradient %d", i);
      if ((rc = check_dev_ptr(tensors[i].grad, name))) return rc;
      snprintf(name, sizeof name, "out of gradient %d", i);
      if (tensors[i].out && tensors[i].out != tensors[i].grad && (rc = check_dev_ptr(tensors[i].out, name))) return rc;
    }
  }
  *grads = g;
  return DISCO_OK;
}

extern "C" size_t disco_grad_workspace_bytes(const disco_grads* grads) {
  if (!grads || grads->count < 0) return 0;
  return (size_t)launches(grads) * kNormGrid * sizeof(Row);
}

extern "C" int disco_grad_norm(const disco_grads* grads, float grad_scale, float* norm, void* workspace,
                               size_t workspace_bytes, void* stream) {
  disco::NvtxScope nvtx_scope("disco_grad_norm");
  int rc;
  if ((rc = check_grads(grads, grad_scale)) || (rc = check_workspace(grads, workspace, workspace_bytes)) ||
      (rc = check_scalar(norm, "norm")) ||
      (rc = check_apart(grads, true, false, norm, workspace, disco_grad_workspace_bytes(grads))))
    return rc;
  return run(grads, grad_scale, 0.0f, false, norm, workspace, (cudaStream_t)stream);
}

extern "C" int disco_grad_clip(const disco_grads* grads, float grad_scale, float max_norm, const float* norm,
                               void* stream) {
  disco::NvtxScope nvtx_scope("disco_grad_clip");
  int rc;
  if ((rc = check_grads(grads, grad_scale)) || (rc = check_max_norm(grads, max_norm)) || (rc = check_scalar(norm, "norm")) ||
      (rc = check_apart(grads, false, true, norm, nullptr, 0)))
    return rc;
  // the kernel writes the norm only where it computes it
#define CALL(N) clip_all<N>(grads, nullptr, 0, grad_scale, max_norm, const_cast<float*>(norm), (cudaStream_t)stream)
  return DISCO_BY_COUNT(grads->count, CALL);
#undef CALL
}

extern "C" int disco_grad_norm_clip(const disco_grads* grads, float grad_scale, float max_norm, float* norm,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  disco::NvtxScope nvtx_scope("disco_grad_norm_clip");
  int rc;
  if ((rc = check_grads(grads, grad_scale)) || (rc = check_max_norm(grads, max_norm)) ||
      (rc = check_workspace(grads, workspace, workspace_bytes)) || (rc = check_scalar(norm, "norm")) ||
      (rc = check_apart(grads, true, true, norm, workspace, disco_grad_workspace_bytes(grads))))
    return rc;
  return run(grads, grad_scale, max_norm, true, norm, workspace, (cudaStream_t)stream);
}
