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
constexpr size_t kStaticSmem = 1024;  // at most, of the kernels of rows; those of tiles have none

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

__device__ __forceinline__ uint4 operator&(uint4 a, uint4 b) { return make_uint4(a.x & b.x, a.y & b.y, a.z & b.z, a.w & b.w); }

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
// word l holds the elements from l V - m on, and a row's first and last words
// are shared with its neighbours in memory.

// Stores words of a row that starts m elements past the aligned address `p` (element
// `first` of a tensor of `total`): n elements of it (the same for the whole warp), of which this lane holds word lx.
// All lanes of the warp call it; rows with `valid` false are not stored.  In a
// full tile, n = (LX - 1) V, the V elements in words that another tile shares
// (the row's first V - m and last m, words 0 and LX - 1) go out one to a lane.
template <int V, typename W>
__device__ __forceinline__ void store_words(void* p, long long first, long long total, W word, int m, int lx, int LX, int n,
                                            bool valid) {
  constexpr int ES = (int)sizeof(W) / V, NW = (int)sizeof(W) / 4;
  const int at = lx * V - m;  // the word's first element in the row
  char* d = (char*)p + lx * (int)sizeof(W);
  if (valid && at >= 0 && at + V <= n && DISCO_IN_BOUNDS(first + m >= 0 && first + lx * V + V <= total)) store_stream(d, word);
  if (n == (LX - 1) * V && LX >= V) {
    uint32_t w[NW];
    memcpy(w, &word, sizeof(W));
    const int e = lx & (V - 1), from = e < m ? LX - 1 : 0;
    uint32_t v = 0;
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      const uint32_t o = __shfl_sync(0xffffffffu, w[k], from, LX);
      v = e * ES / 4 == k ? o : v;
    }
    v >>= 8 * (e * ES & 3);
    if (valid && m > 0 && lx < V && DISCO_IN_BOUNDS(first + from * V + e >= 0 && first + from * V + e < total)) {
      typename Word<ES>::type one;
      memcpy(&one, &v, ES);
      store_stream((char*)p + (from * V + e) * ES, one);
    }
  } else if (valid && at < n && at + V > 0 && !(at >= 0 && at + V <= n)) {
    const uint8_t* b = (const uint8_t*)&word;
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (at + e >= 0 && at + e < n && DISCO_IN_BOUNDS(first + m + at + e >= 0 && first + m + at + e < total)) {
        typename Word<ES>::type v;
        memcpy(&v, b + e * ES, ES);
        store_stream(d + e * ES, v);
      }
  }
}

// ---- asynchronous copies ---------------------------------------------------
// A thread copies only what it reads itself, so its own wait orders them.

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
// of CL CTAs takes it, each CTA cpc channels: thread (lx, j) holds word lx (16
// bytes, V pixels) of the rows of NCH channels.  CTAs are persistent: cluster k
// takes tiles k, k + clusters, ...
// V divides P: TP = LX * V, thread j's channels are j * NCH and the next ones.
// Else (shifted) words are not pixels: the LX words of a row cover TP = (LX - 1) V
// pixels and parts of two neighbouring tiles'.  A thread's channels lie `apart`
// = V / gcd(P, V) channels apart, so that its rows have one skew m, and its V sums
// stand for the pixels from lx V - m on: only the sums and factors are realigned,
// in shared memory, once a tile.  (Shifting the words themselves into place took
// 15 instructions for each: gradient of 64 channels, 84 million elements, 195 us;
// 4-byte accesses to whole pixels 170.)

struct Tiling {
  int NT, LX, NCH, V, CL, cpc, TP, apart;
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

// A thread's words of its NCH channels: `slot` in shared memory, fetched a tile
// ahead, and their places in a tensor.
template <typename T, int V, int NCH, bool SHIFT>
struct Lane {
  using W = Raw<T, V>;
  int lx, LX, nc, stride;  // stride: words from one channel to the next in the ring
  int c0, apart;
  long long P, mine, step, total;  // mine: the thread's place in a tile; step: elements from one of its rows to the next
  W* slot;

  static __host__ __device__ size_t words(const Tiling& g) { return (size_t)NCH * g.NT; }

  __device__ __forceinline__ Lane(const Tiling& g, int B, int C, long long P_, int lx_, int j, int first_c, void* smem)
      : lx(lx_), LX(g.LX), stride(g.NT), apart(SHIFT ? g.apart : 1), P(P_) {
    c0 = first_c + (SHIFT ? j / apart * (apart * NCH) + j % apart : j * NCH);
    const int end = first_c + g.cpc < C ? first_c + g.cpc : C, room = (end - c0 + apart - 1) / apart;
    nc = end <= c0 ? 0 : room < NCH ? room : NCH;
    mine = c0 * P + (SHIFT ? 0 : lx * V);
    step = apart * P;
    total = (long long)B * C * P;
    slot = (W*)smem + threadIdx.x;
  }
  __device__ __forceinline__ int channel(int i) const { return c0 + i * apart; }
  // elements past a word boundary at which the thread's rows start
  __device__ __forceinline__ int skew(const Cursor& c) const { return SHIFT ? (int)((unsigned)(c.off + mine) & (V - 1)) : 0; }
  // whether element e is one of the tile's n pixels
  __device__ __forceinline__ bool in(int e, int m, int n) const {
    const int px = lx * V - m + e;
    return px < n && (!SHIFT || px >= 0);
  }
  // Ones in the bits of a word's elements that are the tile's: the others are
  // another tile's, another row's, or nothing, and may be NaN.
  __device__ __forceinline__ uint4 mask(int m, int n) const {
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      if constexpr (sizeof(T) == 2) {
        const uint16_t u = in(e, m, n) ? 0xffffu : 0u;
        memcpy(&t[e], &u, 2);
      } else {
        const uint32_t u = in(e, m, n) ? 0xffffffffu : 0u;
        memcpy(&t[e], &u, 4);
      }
    }
    uint4 r;
    memcpy(&r, t, 16);
    return r;
  }
  __device__ __forceinline__ void fetch(const Tiling& g, const Cursor& c, const T* p, W* to) const {
    if (c.t >= g.tiles) return;
    const int m = skew(c);
    const long long row = c.off + mine - m + (SHIFT ? lx * V : 0);
    if (c.pos + lx * V - m >= P) return;
    // a word that the tensor's end cuts short is near only the last sample's end
    if (!SHIFT || row + (NCH - 1) * step + V <= total) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
        if (i < nc && DISCO_IN_BOUNDS(row >= 0 && row + i * step + V <= total)) copy_async(to + i * stride, p + row + i * step);
    } else {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const long long left = total - (row + i * step);
        if (i < nc && left > 0 && DISCO_IN_BOUNDS(row >= 0))
          copy_async(to + i * stride, p + row + i * step, left >= V ? 16 : (int)left * (int)sizeof(T));
      }
    }
  }
  // after copy_wait
  __device__ __forceinline__ W read(const W* from, int i) const { return from[i * stride]; }
  // channel i's word, packed as `w` (of any element size), to the tile at c, which
  // has n pixels.  Shifted: called by whole warps.
  template <typename WO>
  __device__ __forceinline__ void write(void* p, const Cursor& c, int m, int i, WO w, int n) const {
    constexpr int ES = (int)sizeof(WO) / V;
    char* d = (char*)p + (c.off + mine + i * step - m) * ES;
    if constexpr (SHIFT) store_words<V>(d, c.off + mine + i * step - m, total, w, m, lx, LX, n, i < nc);
    else if (i < nc && lx * V < n && DISCO_IN_BOUNDS(c.off + mine + i * step + V <= total)) store_stream(d, w);
  }
};

// Cuts a call on `es`-byte elements.  False where the channels of a pixel do
// not fit the largest cluster.
bool plan_tiles(int B, int C, long long P, int es, bool forward, Tiling* g);

// Where a thread's pixels and channels lie, and how a tile's sums over the
// channels are joined: each thread's V sums go to shared memory (one row of
// `slots` for each channel lane), S threads to a pixel add the rows up, and one
// of them turns the sums into the NOUT values that every thread then reads back.
// Pixel px has slot px; shifted, the slots stand in V rows of LX + 1 (pixel px at
// row (px + V) mod V), so that the lanes' accesses lie side by side for any skew.
//
// With a cluster that thread pushes its sums to all peers, into the half of
// `box` of this tile's parity, and one cluster barrier a tile suffices: a CTA
// writes that half again two tiles later, after a barrier that its peers reach
// only when they have read it.
template <int V, int NSUM, int NOUT, bool SHIFT>
struct Joiner {
  int NT, LX, slots, CL, tid, lx, j, rows, S_log, pitch;
  uint32_t rank;
  float *red, *out, *box;

  static __host__ __device__ int slots_of(const Tiling& g) { return SHIFT ? V * (g.LX + 1) : V * g.LX; }
  static __host__ __device__ int pitch_of(const Tiling& g) { return (slots_of(g) + 3) / 4 * 4 + 32; }  // at most
  static __host__ __device__ size_t floats(const Tiling& g) {
    return ((size_t)(g.NT / g.LX) * NSUM * pitch_of(g) + (size_t)slots_of(g) * (NOUT + (g.CL > 1 ? 2 * g.CL * NSUM : 0)) + 3) / 4 * 4;
  }
  __device__ __forceinline__ Joiner(const Tiling& g, float* smem, uint32_t rank_)
      : NT(g.NT), LX(g.LX), slots(slots_of(g)), CL(g.CL), tid(threadIdx.x), rank(rank_) {
    lx = tid & (LX - 1);
    rows = NT / LX;
    j = tid / LX;
    S_log = 0;
    while (S_log < 3 && (2 << S_log) <= rows && (slots << S_log) * 2 <= NT) ++S_log;
    pitch = pitch_of(g) - 32 + (32 >> S_log);
    red = smem;
    out = smem + rows * NSUM * pitch_of(g);
    box = out + slots * NOUT;
  }
  __device__ __forceinline__ int slot(int px) const { return SHIFT ? ((px + V) % V) * (LX + 1) + (px + V) / V : px; }
  // this thread's V values, of skew m, in a row of slots
  __device__ __forceinline__ void put(float* p, const F<V>& f, int m) const {
    if constexpr (SHIFT) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int t = e + V - m;
        p[(t & (V - 1)) * (LX + 1) + lx + (t / V)] = f.v[e];
      }
    } else {
      store_row<V>(p + lx * V, f);
    }
  }
  __device__ __forceinline__ F<V> get(const float* p, int m) const {
    if constexpr (SHIFT) {
      F<V> f;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int t = e + V - m;
        f.v[e] = p[(t & (V - 1)) * (LX + 1) + lx + (t / V)];
      }
      return f;
    } else {
      return load_row<V>(p + lx * V);
    }
  }
  // Hands in this thread's sums.  finish(z, r): the outputs r[NOUT] of one pixel
  // from its sums z[NSUM].  The outputs are there after collect(); what a thread
  // does in between hides the exchange.
  template <typename Fin>
  __device__ __forceinline__ void submit(const F<V> (&s)[NSUM], int m, int parity, Fin finish) const {
#pragma unroll
    for (int n = 0; n < NSUM; ++n) put(red + (n * rows + j) * pitch, s[n], m);
    __syncthreads();
    float* half = box + parity * CL * NSUM * slots;
    const int S = 1 << S_log, part = tid & (S - 1);
    for (int px = tid >> S_log, q0 = 0; q0 < (slots << S_log); q0 += NT, px += NT >> S_log) {
      float z[NSUM], o[NOUT];
#pragma unroll
      for (int n = 0; n < NSUM; ++n) {
        z[n] = 0.0f;
        if (px < slots) {
          const float* p = red + (n * rows + part) * pitch + px;
#pragma unroll 4
          for (int k = part; k < rows; k += S, p += S * pitch) z[n] += *p;
        }
        for (int k = S / 2; k; k >>= 1) z[n] += __shfl_xor_sync(0xffffffffu, z[n], k);
      }
      if (px < slots && part == 0) {
        if (CL == 1) {
          finish(z, o);
#pragma unroll
          for (int n = 0; n < NOUT; ++n) out[n * slots + px] = o[n];
        } else {
#pragma unroll
          for (int n = 0; n < NSUM; ++n)
            for (int k = 0; k < CL; ++k) peer_store(peer(half + (rank * NSUM + n) * slots + px, k), z[n]);
        }
      }
    }
    if (CL > 1) cluster_arrive();
  }
  template <typename Fin>
  __device__ __forceinline__ void collect(F<V> (&r)[NOUT], int m, int parity, Fin finish) const {
    if (CL > 1) {
      cluster_wait();
      const float* half = box + parity * CL * NSUM * slots;
      for (int px = tid; px < slots; px += NT) {
        float z[NSUM], o[NOUT];
#pragma unroll
        for (int n = 0; n < NSUM; ++n) {
          z[n] = 0.0f;
          for (int k = 0; k < CL; ++k) z[n] += half[(k * NSUM + n) * slots + px];
        }
        finish(z, o);
#pragma unroll
        for (int n = 0; n < NOUT; ++n) out[n * slots + px] = o[n];
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NOUT; ++n) r[n] = get(out + n * slots, m);
  }
};

// ---- general kernels: any shape ----------------------------------------------
// A CTA of 8 warps takes 32 pixels, one to a lane, and deals the channels to its
// warps; ROW (P = 1): one row, the channels dealt to its 256 threads.

constexpr int kGenWarps = 8;

template <bool ROW>
struct Dealt {
  static constexpr int PX = ROW ? 1 : 32, STEP = ROW ? kGenWarps * 32 : kGenWarps;  // pixels of a tile; channel step
  static __device__ __forceinline__ int pixel() { return ROW ? 0 : threadIdx.x & 31; }
  static __device__ __forceinline__ int first() { return ROW ? threadIdx.x : threadIdx.x / 32; }
  // over the threads of a pixel
  template <typename Op>
  static __device__ __forceinline__ float join(float v, float (*buf)[32], Op op) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (ROW)
      for (int m = 16; m; m >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, m));
    __syncthreads();
    buf[warp][lane] = v;
    __syncthreads();
    v = buf[0][lane];
    for (int i = 1; i < kGenWarps; ++i) v = op(v, buf[i][lane]);
    return v;
  }
};

__device__ __forceinline__ void let_next_begin() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- launches ----------------------------------------------------------------

// after: the kernel may begin while the one before it on the stream ends, once
// all its CTAs have called let_next_begin(); it calls wait_for_previous() before
// it reads what that one wrote.
// most: the dynamic shared memory that any launch of this kernel may ask for.  The
// limit set on a kernel is shared by all host threads: set to what one call needs,
// it would refuse another thread's larger launch.
template <typename K, typename... A>
int launch(K kernel, int grid, int threads, int cluster, bool after, size_t smem, size_t most, cudaStream_t st,
           const char* what, A... args) {
  if (smem > most) return fail(DISCO_ERR_UNSUPPORTED, "%s: %zu bytes of shared memory", what, smem);
  if (smem + kStaticSmem > 48 * 1024 &&
      cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most) != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(DISCO_ERR_CUDA, "%s: shared memory of %zu bytes refused", what, most);
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
  return launch(kernel, g.clusters * g.CL, g.NT, g.CL, false, smem, kMaxSmem, st, what, args...);
}
template <typename K, typename... A>
int launch_grid(K kernel, int grid, int threads, size_t smem, cudaStream_t st, const char* what, A... args) {
  return launch(kernel, grid, threads, 1, false, smem, kMaxSmem - kStaticSmem, st, what, args...);
}

// ---- arguments, and the kernels by translation unit ---------------------------

struct NormArgs {
  const void *x, *res, *w;
  void *h, *y, *q;
  float* scale;
  float eps, inv_C;
  int G, NG, B, C;
  long long P;
};

struct NormBwdArgs {
  const void *dy, *h, *w, *dh;
  void* dx;
  float* part;  // rows of fp32 partial sums of dweight, or null
  float eps, inv_C;
  int B, C;
  long long P;
};

// 1 / sqrt(mean + eps) from the sum of squares, within 3 ulp; 0 for an infinite sum
__device__ __forceinline__ float inverse_rms(float sum, float inv_C, float eps) { return rsqrtf(fmaf(sum, inv_C, eps)); }

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;  // group maximum of an all-zero group: its scale stays above 0

// DISCO_ERR_UNSUPPORTED, without launching, for shapes the tiles do not take.
int norm_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st);       // without q (disco_norm_tile.cu)
int norm_q_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st);     // with q (disco_norm_q.cu)

int norm_q_any_by_tiles(const NormArgs& a, const Tiling& g, disco_dtype dtype, cudaStream_t st);  // groups of any size
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
