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

// V e4m3 values
template <int V>
__device__ __forceinline__ F<V> unpack_e4m3(const typename Word<V>::type& raw) {
  __nv_fp8x2_storage_t t[V / 2];
  memcpy(t, &raw, V);
  F<V> r;
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    const __half2_raw p = __nv_cvt_fp8x2_to_halfraw2(t[e / 2], __NV_E4M3);  // exact: fp16 holds every e4m3 value
    const float2 f = __half22float2(__half2(p));
    r.v[e] = f.x, r.v[e + 1] = f.y;
  }
  return r;
}

// Each tensor is read once and written once: streaming (evict-first) access.
template <typename W>
__device__ __forceinline__ W load_stream(const void* p) { return __ldcs((const W*)p); }
template <typename W>
__device__ __forceinline__ void store_stream(void* p, W w) { __stcs((W*)p, w); }

// ---- rows off alignment ------------------------------------------------------
// Where V does not divide P a row of V-element words starts m = 0 .. V-1
// elements past a word boundary.  The lanes of a row then move aligned words:
// lane l's elements are the window of words l and l + 1 that starts at element
// m, and word l of an output holds the last m elements of lane l - 1 and the
// first V - m of lane l.

// the word that starts `bytes` (0 .. sizeof(W) - 1) into the pair (a, b)
__device__ __forceinline__ uint32_t window(uint32_t a, uint32_t b, int bytes) { return __funnelshift_r(a, b, 8 * bytes); }
__device__ __forceinline__ uint2 window(uint2 a, uint2 b, int bytes) {
  uint32_t w0 = a.x, w1 = a.y, w2 = b.x;
  if (bytes & 4) w0 = a.y, w1 = b.x, w2 = b.y;
  const int s = 8 * (bytes & 3);
  return make_uint2(__funnelshift_r(w0, w1, s), __funnelshift_r(w1, w2, s));
}
__device__ __forceinline__ uint4 window(uint4 a, uint4 b, int bytes) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (bytes & 8)
#pragma unroll
    for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
  if (bytes & 4)
#pragma unroll
    for (int k = 0; k < 5; ++k) w[k] = w[k + 1];
  const int s = 8 * (bytes & 3);
  return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s),
                    __funnelshift_r(w[3], w[4], s));
}
__device__ __forceinline__ uint32_t from_lane_above(uint32_t v) { return __shfl_down_sync(0xffffffffu, v, 1); }
__device__ __forceinline__ uint2 from_lane_above(uint2 v) { return make_uint2(from_lane_above(v.x), from_lane_above(v.y)); }
__device__ __forceinline__ uint32_t from_lane_below(uint32_t v) { return __shfl_up_sync(0xffffffffu, v, 1); }
__device__ __forceinline__ uint2 from_lane_below(uint2 v) { return make_uint2(from_lane_below(v.x), from_lane_below(v.y)); }
__device__ __forceinline__ uint4 from_lane_below(uint4 v) {
  return make_uint4(from_lane_below(v.x), from_lane_below(v.y), from_lane_below(v.z), from_lane_below(v.w));
}

// Stores the row that starts m elements past the aligned address `p`, `n`
// elements of it (the same for the whole warp), of which this lane holds the V
// from lx * V on.  All lanes of the warp call it; the last of a row's LX lanes
// holds no elements, rows with `valid` false are not stored.  In a full tile,
// n = (LX - 1) V, the V elements that share a word with another tile (the row's
// first V - m and last m) go out one to a lane.
template <int V, typename W>
__device__ __forceinline__ void store_shifted(void* p, W own, int m, int lx, int LX, int n, bool valid) {
  constexpr int ES = (int)sizeof(W) / V, NW = (int)sizeof(W) / 4;
  const W below = from_lane_below(own);
  const W word = m ? window(below, own, (V - m) * ES) : own;
  const int at = lx * V - m;  // the word's first element in the row
  char* d = (char*)p + lx * (int)sizeof(W);
  if (valid && at >= 0 && at + V <= n) store_stream(d, word);
  if (n == (LX - 1) * V && LX >= V) {
    uint32_t own32[NW];
    memcpy(own32, &own, sizeof(W));
    const int e = lx & (V - 1), from = e < V - m ? 0 : LX - 2;
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const uint32_t o = __shfl_sync(0xffffffffu, own32[k], from, LX);
      v = e * ES / 4 == k ? o : v;
    }
    v >>= 8 * (e * ES & 3);
    if (valid && m > 0 && lx < V) {
      const typename Word<ES>::type one = (typename Word<ES>::type)v;
      store_stream((char*)p + (m + from * V + e) * ES, one);
    }
  } else if (valid && at < n && at + V > 0 && !(at >= 0 && at + V <= n)) {
    const uint8_t* b = (const uint8_t*)&word;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (at + e >= 0 && at + e < n) {
        typename Word<ES>::type v;
        memcpy(&v, b + e * ES, ES);
        store_stream(d + e * ES, v);
      }
  }
}

// ---- asynchronous copies ---------------------------------------------------
// A thread copies only what it reads itself (what its warp reads, where rows
// are shifted), so its own wait (and the warp's) orders them.

// 16 bytes, the first `bytes` of them from memory and zeros behind them
__device__ __forceinline__ void copy_async(void* smem, const void* gmem, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(smem))),
               "l"(gmem), "r"(bytes)
               : "memory");
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_barrier() {
  cluster_arrive();
  cluster_wait();
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

// V neighbouring floats of shared memory
template <int V>
__device__ __forceinline__ F<V> load_row(const float* p) {
  F<V> r;
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + e);
      r.v[e] = q.x, r.v[e + 1] = q.y, r.v[e + 2] = q.z, r.v[e + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) r.v[e] = p[e];
  }
  return r;
}
template <int V>
__device__ __forceinline__ void store_row(float* p, const F<V>& f) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 4)
      *reinterpret_cast<float4*>(p + e) = make_float4(f.v[e], f.v[e + 1], f.v[e + 2], f.v[e + 3]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) p[e] = f.v[e];
  }
}

// ---- tiles -----------------------------------------------------------------
// A tile is TP neighbouring pixels of one sample with all channels.  A cluster
// of CL CTAs takes it, each CTA cpc channels: thread (lx, j) holds the V pixels
// from lx * V on (one 16-byte word of each row) of the NCH channels from
// j * NCH on.  CTAs are persistent: cluster k takes tiles k, k + clusters, ...
// V divides P: TP = LX * V.  Else rows are shifted (above), the last lane of a
// row holds no pixels, and TP = (LX - 1) * V.

struct Tiling {
  int NT, LX, NCH, V, CL, cpc, TP;
  int clusters;
  bool shifted;
  long long tiles;             // of the call
  long long span;              // pixels from a sample's first tile to the end of its last
  long long step_b, step_pos;  // what `clusters` tiles on are: samples, and pixels past them
  long long step_off, wrap_off;  // the same in elements; from the end of one sample's tiles to the next sample
  void finish(int B, int C, long long P, long long max_clusters) {
    const long long tpb = (P + TP - 1) / TP;
    tiles = B * tpb;
    clusters = (int)(tiles < max_clusters ? tiles : max_clusters);
    span = tpb * TP;
    step_b = clusters / tpb;
    step_pos = clusters % tpb * TP;
    step_off = step_b * C * P + step_pos;
    wrap_off = (long long)C * P - span;
  }
};

// The tile a cluster is at: its number, sample, first pixel, and the element
// offset of that pixel in the sample's first channel.
struct Cursor {
  long long t, b, pos, off;
  __device__ __forceinline__ Cursor(const Tiling& g, int C, long long P, long long first) : t(first) {
    const long long tpb = g.span / g.TP;
    b = first / tpb;
    pos = (first - b * tpb) * g.TP;
    off = b * C * P + pos;
  }
  __device__ __forceinline__ void next(const Tiling& g) {
    t += g.clusters;
    b += g.step_b;
    pos += g.step_pos;
    off += g.step_off;
    if (pos >= g.span) pos -= g.span, off += g.wrap_off, ++b;
  }
};

// A thread's words of its NCH channels: `ring` in shared memory, fetched a
// tile ahead, and the same places of a tensor.
template <typename T, int V, int NCH, bool SHIFT>
struct Lane {
  using W = Raw<T, V>;
  int lx, LX, nc, stride;  // stride: words from one channel to the next in the ring
  int c0;
  long long P, mine, total;  // mine: the thread's place in a tile; total: elements of the tensor
  W* slot;

  static __host__ __device__ size_t words(const Tiling& g) { return (size_t)NCH * g.NT + (SHIFT ? 1 : 0); }

  __device__ __forceinline__ Lane(const Tiling& g, int B, int C, long long P_, int lx_, int j, int first_c, void* smem)
      : lx(lx_), LX(g.LX), stride(g.NT), P(P_) {
    c0 = first_c + j * NCH;
    const int end = first_c + g.cpc < C ? first_c + g.cpc : C;
    nc = end - c0 < 0 ? 0 : end - c0 < NCH ? end - c0 : NCH;
    mine = c0 * P + (SHIFT ? 0 : lx * V);
    total = (long long)B * C * P;
    slot = (W*)smem + threadIdx.x;
  }
  // pixels of this thread in the tile at c: 0 .. V
  __device__ __forceinline__ int pixels(const Tiling& g, const Cursor& c) const {
    if (c.t >= g.tiles) return 0;
    const long long n = P - c.pos - lx * V;
    if constexpr (SHIFT) return lx == g.LX - 1 || n <= 0 ? 0 : n < V ? (int)n : V;
    else return n > 0 ? V : 0;
  }
  // elements past a word boundary at which the row of channel i starts
  __device__ __forceinline__ int skew(const Cursor& c, int i) const {
    return SHIFT ? (int)((unsigned)(c.off + mine + i * P) & (V - 1)) : 0;
  }
  __device__ __forceinline__ void fetch(const Tiling& g, const Cursor& c, const T* p, W* to) const {
    if (c.t >= g.tiles) return;
    if constexpr (SHIFT) {
      const T* q = p + lx * V;
      // every word of the tile within its row, and none near the tensor's end
      if (c.pos + LX * V <= P && c.off + mine + NCH * P + (LX + 1) * V <= total) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          const long long row = (c.off + mine + i * P) & ~(long long)(V - 1);
          if (i < nc && DISCO_IN_BOUNDS(row >= 0)) copy_async(to + i * stride, q + row);
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const long long row = c.off + mine + i * P;
        const int m = (int)((unsigned)row & (V - 1));
        const long long at = row - m + lx * V;
        if (i < nc && c.pos + lx * V - m < P && at < total && DISCO_IN_BOUNDS(at >= 0))
          copy_async(to + i * stride, p + at, total - at >= V ? 16 : (int)(total - at) * (int)sizeof(T));
      }
    } else if (c.pos + lx * V < P) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc && DISCO_IN_BOUNDS(c.off + mine >= 0 && c.off + mine + i * P + V <= total))
          copy_async(to + i * stride, p + c.off + mine + i * P);
    }
  }
  // after copy_wait (and __syncwarp, if shifted)
  __device__ __forceinline__ W read(const W* from, int i, int m) const {
    const W w = from[i * stride];
    if constexpr (SHIFT) return window(w, from[i * stride + 1], m * (int)sizeof(T));
    return w;
  }
  // channel i's V elements, packed as `w` (of any element size), to the tile at
  // c; n: pixels of the row in the tile.  Shifted: called by whole warps.
  template <typename WO>
  __device__ __forceinline__ void write(void* p, const Cursor& c, int i, WO w, bool on, int n) const {
    constexpr int ES = (int)sizeof(WO) / V;
    const long long row = c.off + mine + i * P;
    if constexpr (SHIFT) {
      const int m = (int)((unsigned)row & (V - 1));
      store_shifted<V>((char*)p + (row & ~(long long)(V - 1)) * ES, w, m, lx, LX, n, i < nc);
    } else {
      if (on && i < nc && DISCO_IN_BOUNDS(row >= 0 && row + V <= total)) store_stream((char*)p + row * ES, w);
    }
  }
};

// Cuts a call on `es`-byte elements.  False where the channels of a pixel do
// not fit the largest cluster.
bool plan_tiles(int B, int C, long long P, int es, bool forward, Tiling* g);

// Where a thread's pixels and channels lie, and how a tile's sums over the
// channels are joined: each thread's V sums go to shared memory (one row for
// each channel lane), S threads to a pixel add the rows up, and one of them
// turns the sums into the NOUT values that every thread then reads back.
//
// With a cluster that thread pushes its sums to all peers, into the half of
// `box` of this tile's parity, and one cluster barrier a tile suffices: a CTA
// writes that half again two tiles later, after a barrier that its peers reach
// only when they have read it.
template <int V, int NSUM, int NOUT>
struct Joiner {
  int NT, LX, TP, CL, tid, lx, j, rows, S_log, pitch;
  uint32_t rank;
  float *red, *out, *box;

  static __host__ __device__ size_t floats(const Tiling& g) {
    const int TP = g.LX * V;  // with the pixels of a last lane that holds none
    return (size_t)(g.NT / g.LX) * NSUM * (TP + 32) + (size_t)TP * NOUT + (g.CL > 1 ? 2 * (size_t)g.CL * NSUM * TP : 0);
  }
  __device__ __forceinline__ Joiner(const Tiling& g, float* smem, uint32_t rank_)
      : NT(g.NT), LX(g.LX), TP(g.LX * V), CL(g.CL), tid(threadIdx.x), rank(rank_) {
    lx = tid & (LX - 1);
    rows = NT / LX;
    j = tid / LX;
    S_log = 0;
    while (S_log < 3 && (2 << S_log) <= rows && (TP << S_log) * 2 <= NT) ++S_log;
    pitch = TP + (32 >> S_log);
    red = smem;
    out = smem + rows * NSUM * (TP + 32);
    box = out + TP * NOUT;
  }
  // Hands in this thread's sums.  finish(z, r): the outputs r[NOUT] of one pixel
  // from its sums z[NSUM].  The outputs are there after collect(); what a thread
  // does in between hides the exchange.
  template <typename Fin>
  __device__ __forceinline__ void submit(const F<V> (&s)[NSUM], int parity, Fin finish) const {
#pragma unroll
    for (int n = 0; n < NSUM; ++n) store_row<V>(red + (n * rows + j) * pitch + lx * V, s[n]);
    __syncthreads();
    float* half = box + parity * CL * NSUM * TP;
    const int S = 1 << S_log, part = tid & (S - 1);
    for (int px = tid >> S_log, q0 = 0; q0 < (TP << S_log); q0 += NT, px += NT >> S_log) {
      float z[NSUM], o[NOUT];
#pragma unroll
      for (int n = 0; n < NSUM; ++n) {
        z[n] = 0.0f;
        if (px < TP) {
          const float* p = red + (n * rows + part) * pitch + px;
#pragma unroll 4
          for (int k = part; k < rows; k += S, p += S * pitch) z[n] += *p;
        }
        for (int m = S / 2; m; m >>= 1) z[n] += __shfl_xor_sync(0xffffffffu, z[n], m);
      }
      if (px < TP && part == 0) {
        if (CL == 1) {
          finish(z, o);
#pragma unroll
          for (int n = 0; n < NOUT; ++n) out[n * TP + px] = o[n];
        } else {
#pragma unroll
          for (int n = 0; n < NSUM; ++n)
            for (int k = 0; k < CL; ++k) peer_store(peer(half + (rank * NSUM + n) * TP + px, k), z[n]);
        }
      }
    }
    if (CL > 1) cluster_arrive();
  }
  template <typename Fin>
  __device__ __forceinline__ void collect(F<V> (&r)[NOUT], int parity, Fin finish) const {
    if (CL > 1) {
      cluster_wait();
      const float* half = box + parity * CL * NSUM * TP;
      for (int px = tid; px < TP; px += NT) {
        float z[NSUM], o[NOUT];
#pragma unroll
        for (int n = 0; n < NSUM; ++n) {
          z[n] = 0.0f;
          for (int k = 0; k < CL; ++k) z[n] += half[(k * NSUM + n) * TP + px];
        }
        finish(z, o);
#pragma unroll
        for (int n = 0; n < NOUT; ++n) out[n * TP + px] = o[n];
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NOUT; ++n) r[n] = load_row<V>(out + n * TP + lx * V);
  }
};

// ---- general kernels: 32 pixels per CTA, the channels dealt to 8 warps ------

constexpr int kGenWarps = 8;

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
__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- launches ----------------------------------------------------------------

// after: the kernel may begin while the one before it on the stream ends, once
// all its CTAs have called let_next_begin(); it calls wait_for_previous() before
// it reads what that one wrote.
template <typename K, typename... A>
int launch(K kernel, int grid, int threads, int cluster, bool after, size_t smem, cudaStream_t st, const char* what, A... args) {
  if (smem + 1024 > 48 * 1024 &&  // with a kernel's static arrays
      cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DISCO_ERR_CUDA, "%s: shared memory of %zu bytes refused", what, smem);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)cluster;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  if (after) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DISCO_ERR_LAUNCH, "%s: %s", what, cudaGetErrorString(e));
  }
  return DISCO_OK;
}
template <typename K, typename... A>
int launch_clusters(K kernel, const Tiling& g, size_t smem, cudaStream_t st, const char* what, A... args) {
  return launch(kernel, g.clusters * g.CL, g.NT, g.CL, false, smem, st, what, args...);
}
template <typename K, typename... A>
int launch_grid(K kernel, int grid, int threads, size_t smem, cudaStream_t st, const char* what, A... args) {
  return launch(kernel, grid, threads, 1, false, smem, st, what, args...);
}

// ---- arguments, and the kernels by translation unit ---------------------------

struct NormArgs {
  const void *x, *res, *w;
  void *h, *y, *q;
  float* scale;
  float eps;
  int G, NG, B, C;
  long long P;
};

struct NormBwdArgs {
  const void *dy, *h, *w, *dh;
  void* dx;
  float* part;  // rows of fp32 partial sums of dweight, or null
  float eps;
  int B, C;
  long long P;
};

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;  // group maximum of an all-zero group: its scale stays above 0

// DISCO_ERR_UNSUPPORTED, without launching, for shapes the tiles do not take.
int norm_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st);       // without q (disco_norm_tile.cu)
int norm_q_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st);     // with q (disco_norm_q.cu)

int norm_by_rows(const NormArgs& a, disco_dtype dtype, cudaStream_t st);        // P = 1 (disco_norm_rows.cu)
int norm_bwd_by_rows(const NormBwdArgs& a, disco_dtype dtype, cudaStream_t st);
int norm_bwd_rows_parts(int B, int C, int es);  // rows of partial sums of that call, 0: not taken

// ---- host checks (disco_norm.cu) -------------------------------------------

struct Buffer {
  const void* p;
  size_t bytes;
  const char* name;
};
int check_buffers(const Buffer* in, const unsigned* in_place, int nin, const Buffer* out, int nout);
int check_shape(int32_t B, int32_t C, int64_t P, disco_dtype dtype);
int check_eps(float eps);
// groups of a pixel's channels; *G: channels of one
inline int groups(int32_t C, int32_t group, int* G) {
  *G = group > 0 && group < C ? group : C;
  return (C + *G - 1) / *G;
}
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
