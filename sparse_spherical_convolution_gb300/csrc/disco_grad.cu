// disco_grad.cu -- the Euclidean norm over all gradients of a model and their
// scaling to a largest norm (disco_grad_norm, disco_grad_clip).
//
// The list of gradients travels in the kernels' parameters, so a call depends
// on no device table and no earlier copy.  Work is cut into chunks of
// kChunk elements that do not cross tensors; a CTA takes chunks blockIdx.x,
// blockIdx.x + gridDim.x, ...
//
// Sums of squares are kept at three scales, sum g^2, sum (g 2^-80)^2 and
// sum (g 2^90)^2: where the first is infinite the second holds the answer,
// where it is below 2^-60 (its terms near the smallest fp32) the third.

#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "disco_bounds.cuh"
#include "disco_internal.cuh"

namespace disco {

DISCO_BOUNDS_READER(grad_bounds)

namespace {

constexpr int kChunk = 4096;
constexpr int kThreads = 256;
constexpr int kGrid = 304;       // CTAs of a norm launch = rows of its partial sums
constexpr int kMaxTensors = 256; // gradients of one launch

struct Entry {
  const void* g;
  void* o;
  long long n;
  long long chunk0;  // first chunk of the tensor
  int dt, odt;
};
struct Table {
  Entry e[kMaxTensors];
  long long chunks;
  int count;
};

__device__ __forceinline__ float load_as_f32(const void* p, long long i, int dt) {
  if (dt == DISCO_F32) return ((const float*)p)[i];
  if (dt == DISCO_BF16) return to_f32(((const __nv_bfloat16*)p)[i]);
  return to_f32(((const __half*)p)[i]);
}
__device__ __forceinline__ void store_f32(void* p, long long i, int dt, float v) {
  if (dt == DISCO_F32) ((float*)p)[i] = v;
  else if (dt == DISCO_BF16) ((__nv_bfloat16*)p)[i] = from_f32<__nv_bfloat16>(v);
  else ((__half*)p)[i] = from_f32<__half>(v);
}

// the tensor that chunk c belongs to
__device__ __forceinline__ int find(const Table& t, long long c) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.e[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Table t, double* part) {
  float a = 0.0f, b = 0.0f, c = 0.0f;
  for (long long k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const Entry& e = t.e[find(t, k)];
    const long long i0 = (k - e.chunk0) * kChunk, i1 = min(e.n, i0 + kChunk);
    for (long long i = i0 + threadIdx.x; i < i1; i += kThreads) {
      const float v = load_as_f32(e.g, i, e.dt);
      const float u = v * 0x1p-80f, w = v * 0x1p90f;
      a = fmaf(v, v, a);
      b = fmaf(u, u, b);
      c = fmaf(w, w, c);
    }
  }
  __shared__ double s[3][kThreads];
  s[0][threadIdx.x] = a;
  s[1][threadIdx.x] = b;
  s[2][threadIdx.x] = c;
  for (int m = kThreads / 2; m; m >>= 1) {
    __syncthreads();
    if (threadIdx.x < m)
      for (int j = 0; j < 3; ++j) s[j][threadIdx.x] += s[j][threadIdx.x + m];
  }
  if (threadIdx.x < 3) part[(long long)blockIdx.x * 3 + threadIdx.x] = s[threadIdx.x][0];
}

__global__ void grad_norm_finish_kernel(const double* part, int parts, float grad_scale, float* norm) {
  double s[3] = {0.0, 0.0, 0.0};
  for (int i = 0; i < parts; ++i)
    for (int j = 0; j < 3; ++j) s[j] += part[(long long)i * 3 + j];
  double v = sqrt(s[0]);
  if (isinf(s[0])) v = sqrt(s[1]) * 0x1p80;
  else if (s[0] < 0x1p-60) v = sqrt(s[2]) * 0x1p-90;
  *norm = (float)(v * grad_scale);
}

__global__ void __launch_bounds__(kThreads)
    grad_clip_kernel(const __grid_constant__ Table t, float grad_scale, float max_norm, const float* norm) {
  const float n = *norm;
  const float f = n <= max_norm ? grad_scale : grad_scale * (max_norm / n);
  for (long long k = blockIdx.x; k < t.chunks; k += gridDim.x) {
    const Entry& e = t.e[find(t, k)];
    if (e.o == e.g && f == 1.0f) continue;
    const long long i0 = (k - e.chunk0) * kChunk, i1 = min(e.n, i0 + kChunk);
    for (long long i = i0 + threadIdx.x; i < i1; i += kThreads)
      store_f32(e.o, i, e.odt, load_as_f32(e.g, i, e.dt) * f);
  }
}

// Fills `t` from tensors[*next ...]; false when none with elements is left.
bool fill(const disco_grads* g, int* next, Table* t) {
  t->count = 0;
  t->chunks = 0;
  for (; *next < g->count && t->count < kMaxTensors; ++*next) {
    const disco_grad_tensor& s = g->tensors[*next];
    if (s.n < 1) continue;
    t->e[t->count++] = Entry{s.grad, s.out, s.n, t->chunks, s.dtype, s.out_dtype};
    t->chunks += (s.n + kChunk - 1) / kChunk;
  }
  return t->count > 0;
}

int launches(const disco_grads* g) { return g->count / kMaxTensors + 1; }

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

int run_norm(const disco_grads* g, float grad_scale, float* norm, void* ws, cudaStream_t st) {
  Table t;
  int next = 0, parts = 0;
  double* part = (double*)ws;
  while (fill(g, &next, &t)) {
    const int grid = (int)(t.chunks < kGrid ? t.chunks : kGrid);
    grad_norm_kernel<<<grid, kThreads, 0, st>>>(t, part + 3LL * parts);
    parts += grid;
  }
  grad_norm_finish_kernel<<<1, 1, 0, st>>>(part, parts, grad_scale, norm);
  return check_launch("grad_norm_kernel");
}

int run_clip(const disco_grads* g, float grad_scale, float max_norm, const float* norm, cudaStream_t st) {
  Table t;
  int next = 0;
  while (fill(g, &next, &t)) {
    const int grid = (int)(t.chunks < kGrid * 4 ? t.chunks : kGrid * 4);
    grad_clip_kernel<<<grid, kThreads, 0, st>>>(t, grad_scale, max_norm, norm);
  }
  return check_launch("grad_clip_kernel");
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
  return (size_t)launches(grads) * kGrid * 3 * sizeof(double);
}

extern "C" int disco_grad_norm(const disco_grads* grads, float grad_scale, float* norm, void* workspace,
                               size_t workspace_bytes, void* stream) {
  disco::NvtxScope nvtx_scope("disco_grad_norm");
  int rc;
  if ((rc = check_grads(grads, grad_scale)) || (rc = check_workspace(grads, workspace, workspace_bytes)) ||
      (rc = check_scalar(norm, "norm")))
    return rc;
  return run_norm(grads, grad_scale, norm, workspace, (cudaStream_t)stream);
}

extern "C" int disco_grad_clip(const disco_grads* grads, float grad_scale, float max_norm, const float* norm,
                               void* stream) {
  disco::NvtxScope nvtx_scope("disco_grad_clip");
  int rc;
  if ((rc = check_grads(grads, grad_scale)) || (rc = check_max_norm(grads, max_norm)) || (rc = check_scalar(norm, "norm")))
    return rc;
  return run_clip(grads, grad_scale, max_norm, norm, (cudaStream_t)stream);
}

extern "C" int disco_grad_norm_clip(const disco_grads* grads, float grad_scale, float max_norm, float* norm,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  disco::NvtxScope nvtx_scope("disco_grad_norm_clip");
  int rc;
  if ((rc = check_grads(grads, grad_scale)) || (rc = check_max_norm(grads, max_norm)) ||
      (rc = check_workspace(grads, workspace, workspace_bytes)) || (rc = check_scalar(norm, "norm")))
    return rc;
  if ((rc = run_norm(grads, grad_scale, norm, workspace, (cudaStream_t)stream))) return rc;
  return run_clip(grads, grad_scale, max_norm, norm, (cudaStream_t)stream);
}
