// disco_norm.cuh -- what the channel norm's kernels share (disco_norm.cu,
// disco_norm_bwd.cu): packed fp32 arithmetic on V neighbouring pixels, typed
// vector access, thread-private asynchronous copies, and how a call is cut
// into tiles.  Not part of the ABI.
#pragma once

#include <cuda_fp8.h>
#include <math.h>
#include <string.h>

#include "disco_bounds.cuh"
#include "disco_internal.cuh"

namespace disco {
namespace norm {

constexpr int kSMs = 152;
constexpr int kMaxThreads = 512;
constexpr size_t kMaxSmem = 227 * 1024;

// ---- V fp32 values, two to an instruction (f32x2) where V is even ---------

template <int V>
struct F {
  float v[V];
};

__device__ __forceinline__ unsigned long long pair(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(unsigned long long r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}

template <int V>
__device__ __forceinline__ F<V> fill(float x) {
  F<V> r;
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = x;
  return r;
}

template <int V>
__device__ __forceinline__ F<V> fma(const F<V>& a, const F<V>& b, const F<V>& c) {
  F<V> r;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      unsigned long long o;
      asm("fma.rn.f32x2 %0, %1, %2, %3;"
          : "=l"(o)
          : "l"(pair(a.v[e], a.v[e + 1])), "l"(pair(b.v[e], b.v[e + 1])), "l"(pair(c.v[e], c.v[e + 1])));
      unpair(o, r.v[e], r.v[e + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = fmaf(a.v[e], b.v[e], c.v[e]);
  }
  return r;
}
template <int V>
__device__ __forceinline__ F<V> mul(const F<V>& a, const F<V>& b) {
  F<V> r;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      unsigned long long o;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(o) : "l"(pair(a.v[e], a.v[e + 1])), "l"(pair(b.v[e], b.v[e + 1])));
      unpair(o, r.v[e], r.v[e + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = a.v[e] * b.v[e];
  }
  return r;
}
template <int V>
__device__ __forceinline__ F<V> add(const F<V>& a, const F<V>& b) {
  F<V> r;
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      unsigned long long o;
      asm("add.rn.f32x2 %0, %1, %2;" : "=l"(o) : "l"(pair(a.v[e], a.v[e + 1])), "l"(pair(b.v[e], b.v[e + 1])));
      unpair(o, r.v[e], r.v[e + 1]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = a.v[e] + b.v[e];
  }
  return r;
}

// ---- V elements of type T as one word ------------------------------------

template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<4> { using type = uint32_t; };
template <> struct Word<2> { using type = uint16_t; };
template <> struct Word<1> { using type = uint8_t; };

template <typename T, int V>
using Raw = typename Word<(int)sizeof(T) * V>::type;

template <typename T, int V>
__device__ __forceinline__ F<V> unpack(const Raw<T, V>& raw) {
  F<V> r;
  T t[V];
  memcpy(t, &raw, sizeof(raw));
#pragma unroll
  for (int e = 0; e < V; ++e) r.v[e] = to_f32(t[e]);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> packed(const F<V>& f) {
  T t[V];
  if constexpr (V % 2 == 0 && sizeof(T) == 2) {  // one conversion for two elements
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      if constexpr (__is_same(T, __nv_bfloat16)) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(f.v[e], f.v[e + 1]);
        t[e] = p.x, t[e + 1] = p.y;
      } else {
        const __half2 p = __floats2half2_rn(f.v[e], f.v[e + 1]);
        t[e] = p.x, t[e + 1] = p.y;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = from_f32<T>(f.v[e]);
  }
  Raw<T, V> raw;
  memcpy(&raw, t, sizeof(raw));
  return raw;
}
template <int V>
__device__ __forceinline__ typename Word<V>::type packed_e4m3(const F<V>& f) {
  uint8_t t[V];
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const __nv_fp8x2_storage_t p =
          __nv_cvt_float2_to_fp8x2(make_float2(f.v[e], f.v[e + 1]), __NV_SATFINITE, __NV_E4M3);
      memcpy(t + e, &p, 2);
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = (uint8_t)__nv_cvt_float_to_fp8(f.v[e], __NV_SATFINITE, __NV_E4M3);
  }
  typename Word<V>::type raw;
  memcpy(&raw, t, sizeof(raw));
  return raw;
}

// Each tensor is read once and written once: streaming (evict-first) access.
template <typename W>
__device__ __forceinline__ W load_stream(const void* p) { return __ldcs((const W*)p); }
template <typename W>
__device__ __forceinline__ void store_stream(void* p, W w) { __stcs((W*)p, w); }

// ---- thread-private asynchronous copies ----------------------------------
// A thread copies only what it reads itself, so its own wait orders them and
// no barrier is needed.

template <int BYTES>
__device__ __forceinline__ void copy_async(void* smem, const void* gmem) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(gmem) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(gmem), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// ---- thread-block clusters ------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// address of `p` (this CTA's shared memory) in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_store(uint32_t a, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}
__device__ __forceinline__ uint32_t peer_load(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// ---- tiles -----------------------------------------------------------------
// A tile is TP = LX * V neighbouring pixels of one sample with all channels.
// A cluster of CL CTAs takes it, each CTA cpc channels: thread (lx, j) holds
// V pixels of the NCH channels from j * NCH on.  CTAs are persistent: cluster
// k takes tiles k, k + clusters, ...

struct Tiling {
  int NT, LX, NCH, V, CL, cpc;
  long long tpb, tiles;       // tiles of a sample, of the call
  int clusters;
  long long step_b, step_t;   // clusters = step_b samples and step_t tiles
};

// The tile a cluster is at.
struct Cursor {
  long long t, b, ti;
  __device__ __forceinline__ Cursor(const Tiling& g, long long first) : t(first), b(first / g.tpb), ti(first - b * g.tpb) {}
  __device__ __forceinline__ void next(const Tiling& g) {
    t += g.clusters;
    b += g.step_b;
    ti += g.step_t;
    if (ti >= g.tpb) ti -= g.tpb, ++b;
  }
};

// Cuts a call on `es`-byte elements.  False where
// the channels of a pixel do not fit the largest cluster.  `most`: largest
// number of channels to a thread, as a multiple of the smallest (4 vectors of
// 16 bytes, 8 narrower ones).
bool plan_tiles(int B, int C, long long P, int es, int most, Tiling* g);

// Where a thread's pixels and channels lie, and how a tile's sums are joined.
//
// Sums over channels: in registers over a thread's channels, by shuffles over
// the channel lanes of a warp (LX < 32), then through `rows` rows of shared
// memory, S threads to a pixel; with a cluster each CTA pushes its sums to all
// its peers, into the half of `tot` of this tile's parity, and one cluster
// barrier a tile suffices: a CTA writes that half again two tiles later, after
// a barrier that its peers reach only when they have read it.
template <int V, int NSUM>
struct Joiner {
  int NT, LX, TP, CL, tid, lx, j, rows, row, S, S_log, pitch;
  uint32_t rank;
  float *red, *tot;

  static __host__ __device__ size_t floats(const Tiling& g) {
    const int TP = g.LX * V, rows = g.LX < 32 ? g.NT / 32 : g.NT / g.LX;
    return (size_t)rows * NSUM * (TP + 32) + 2 * (size_t)g.CL * NSUM * TP;
  }
  __device__ __forceinline__ Joiner(const Tiling& g, float* smem, uint32_t rank_)
      : NT(g.NT), LX(g.LX), TP(g.LX * V), CL(g.CL), tid(threadIdx.x), rank(rank_) {
    lx = tid & (LX - 1);
    j = tid / LX;
    rows = LX < 32 ? NT / 32 : NT / LX;
    row = LX < 32 ? tid / 32 : j;
    S_log = 0;
    while (S_log < 3 && (2 << S_log) <= rows && (TP << S_log) * 2 <= NT) ++S_log;
    S = 1 << S_log;
    pitch = TP + 32 / S;
    red = smem;
    tot = smem + rows * NSUM * (TP + 32);
  }
  // s: this thread's sums of its V pixels; returns those over all channels
  __device__ __forceinline__ void join(F<V> (&s)[NSUM], int parity) const {
    for (int m = 16; m >= LX; m >>= 1)
#pragma unroll
      for (int n = 0; n < NSUM; ++n) {
        F<V> o;
#pragma unroll
        for (int e = 0; e < V; ++e) o.v[e] = __shfl_xor_sync(0xffffffffu, s[n].v[e], m);
        s[n] = add(s[n], o);
      }
    if (LX >= 32 || (tid & 31) < LX)
#pragma unroll
      for (int n = 0; n < NSUM; ++n)
#pragma unroll
        for (int e = 0; e < V; ++e) red[(n * rows + row) * pitch + lx * V + e] = s[n].v[e];
    __syncthreads();
    float* t = tot + parity * CL * NSUM * TP;
    for (int q0 = 0; q0 < TP * S; q0 += NT) {
      const int q = q0 + tid, px = q >> S_log, part = q & (S - 1);
#pragma unroll
      for (int n = 0; n < NSUM; ++n) {
        float z = 0.0f;
        if (px < TP)
          for (int k = part; k < rows; k += S) z += red[(n * rows + k) * pitch + px];
        for (int m = S / 2; m; m >>= 1) z += __shfl_xor_sync(0xffffffffu, z, m);
        if (px < TP && part == 0) {
          float* d = t + (rank * NSUM + n) * TP + px;
          if (CL == 1) *d = z;
          else
            for (int k = 0; k < CL; ++k) peer_store(peer(d, k), z);
        }
      }
    }
    if (CL == 1) __syncthreads();
    else cluster_barrier();
#pragma unroll
    for (int n = 0; n < NSUM; ++n) {
      F<V> z = fill<V>(0.0f);
      for (int k = 0; k < CL; ++k)
#pragma unroll
        for (int e = 0; e < V; ++e) z.v[e] += t[(k * NSUM + n) * TP + lx * V + e];
      s[n] = z;
    }
  }
};

// Launches a tile kernel on its clusters.
template <typename K, typename... A>
int launch_clusters(K kernel, const Tiling& g, size_t smem, cudaStream_t st, const char* what, A... args) {
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
    return fail(DISCO_ERR_CUDA, "%s: shared memory of %zu bytes refused", what, smem);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(g.clusters * g.CL));
  cfg.blockDim = dim3((unsigned)g.NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)g.CL;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = g.CL > 1 ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) return fail(DISCO_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
  return check_launch(what);
}

// ---- host checks (disco_norm.cu) -------------------------------------------

struct Buffer {
  const void* p;
  size_t bytes;
  const char* name;
};
int check_buffers(const Buffer* in, const unsigned* in_place, int nin, const Buffer* out, int nout);
int check_shape(int32_t B, int32_t C, int64_t P, disco_dtype dtype);
int check_eps(float eps);
inline int elem_bytes(disco_dtype dt) { return dt == DISCO_F32 ? 4 : 2; }

// CALL(T) for the element type of dtype.
#define DISCO_BY_DTYPE(dtype, CALL)              \
  switch (dtype) {                               \
    case DISCO_F32: CALL(float); break;          \
    case DISCO_BF16: CALL(__nv_bfloat16); break; \
    default: CALL(__half); break;                \
  }

}  // namespace norm
}  // namespace disco
