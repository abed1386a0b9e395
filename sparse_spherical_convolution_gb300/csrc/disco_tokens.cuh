// disco_tokens.cuh -- the kernels that work token by token, each token's values held
// in registers between the join of the largest magnitude and the rounding
// (disco_quant_i8, disco_glu).  Not part of the ABI.
//
// A token's C values are dealt over the threads of one CTA.  On grids a thread
// takes V neighbouring pixels (one 16-byte word, or one pixel where V does not
// divide P) of J channels, NL channels apart; LX threads lie side by side along
// the pixels.  In rows (P = 1) V neighbouring channels, J words.  All loads of a thread
// are in flight at once, many CTAs share an SM, and the largest magnitude crosses the
// CTA by one row of shared memory for each warp: one barrier a tile.
#pragma once

#include "disco_i8.cuh"

namespace disco {
namespace i8 {

using norm::F;
using norm::Raw;
using norm::Word;
using norm::load_stream;
using norm::store_stream;
using norm::unpack;
using norm::packed;

// x [B, C or 2 C, P]; the outputs that are not wanted are null.
struct TokenArgs {
  const void* x;
  void* y;
  int8_t* q;
  float* scale;
  int8_t* xq;
  float* xscale;
  int act, B, C;
  long long P;
};

struct TokenCut {
  int LX, NL, TP;       // threads along pixels, along channels; pixels of a tile
  long long per_sample; // tiles of a sample (grids)
};

constexpr int kTokenThreads = 512;

// magnitudes of a word: two to a register for 16-bit types
template <typename T, int V>
struct Mag {
  static constexpr int N = sizeof(T) == 2 && V > 1 ? V / 2 : V;
  uint32_t m[N];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = 0;
  }
  template <typename W>
  __device__ __forceinline__ void add(const W& w) {
    if constexpr (sizeof(T) == 4) {
      uint32_t t[V];
      memcpy(t, &w, sizeof(w));
#pragma unroll
      for (int i = 0; i < V; ++i) m[i] = max32(m[i], t[i]);
    } else if constexpr (V == 1) {
      m[0] = max(m[0], (uint32_t)w & 0x7fffu);
    } else {
      uint32_t t[V / 2];
      memcpy(t, &w, sizeof(w));
#pragma unroll
      for (int i = 0; i < V / 2; ++i) m[i] = max16(m[i], t[i]);
    }
  }
  __device__ __forceinline__ void join(uint32_t o, int i) {
    if constexpr (sizeof(T) == 2 && V > 1) m[i] = __vmaxu2(m[i], o);
    else m[i] = max(m[i], o);
  }
  __device__ __forceinline__ float value(int e) const {
    if constexpr (sizeof(T) == 4) {
      return __uint_as_float(m[e]);
    } else {
      const uint32_t b = V > 1 ? (m[e / 2] >> (16 * (e & 1))) & 0xffffu : m[0];
      T t;
      const uint16_t h = (uint16_t)b;
      memcpy(&t, &h, 2);
      return to_f32(t);
    }
  }
  __device__ __forceinline__ float all() const {  // the largest of the word's V
    uint32_t r = m[0];
#pragma unroll
    for (int i = 1; i < N; ++i) r = sizeof(T) == 2 && V > 1 ? __vmaxu2(r, m[i]) : max(r, m[i]);
    if constexpr (sizeof(T) == 4) return __uint_as_float(r);
    if (V > 1) r = max(r & 0xffffu, r >> 16);
    T t;
    const uint16_t h = (uint16_t)r;
    memcpy(&t, &h, 2);
    return to_f32(t);
  }
};

template <int V>
__device__ __forceinline__ void store_bytes(int8_t* p, const uint32_t (&r)[V]) {
  typename Word<V>::type o;
  if constexpr (V == 1) {
    o = (uint8_t)r[0];
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) w[i] = bytes4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    memcpy(&o, w, V);
  }
  store_stream(p, o);
}

// GLU: x holds gates and values, 2 C channels; y = act(gate) value.  XQ: the 8-bit
// form of x; YQ: that of y.
template <typename T, int V, int J, bool GLU, bool XQ, bool YQ>
__global__ void __launch_bounds__(kTokenThreads) tokens_tile_kernel(const TokenArgs a, const TokenCut g) {
  constexpr int G = GLU ? 2 : 1;
  using R = Raw<T, V>;
  using MX = Mag<T, V>;
  using MY = Mag<float, V>;
  constexpr int NM = (XQ ? MX::N : 0) + (YQ ? MY::N : 0);
  extern __shared__ uint32_t sums[];  // [warps][NM][LX], or the 32 lanes' where a row of lanes is wider
  const int tid = threadIdx.x, lx = tid & (g.LX - 1), j0 = tid / g.LX;
  const long long t = blockIdx.x, b = t / g.per_sample, p = (t - b * g.per_sample) * g.TP + lx * V;
  const bool live = p < a.P;
  const T* x = (const T*)a.x + b * G * a.C * a.P + p;
  const long long half = a.C * a.P, y0 = b * a.C * a.P + p;
  R w[G][J];
  float y[YQ ? J : 1][V];
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int c = j0 + i * g.NL;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      memset(&w[h][i], 0, sizeof(R));
      if (live && c < a.C && DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) w[h][i] = load_stream<R>(x + h * half + c * a.P);
    }
  }
  MX mx;
  MY my;
  mx.clear(), my.clear();
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int c = j0 + i * g.NL;
    if constexpr (XQ)
#pragma unroll
      for (int h = 0; h < G; ++h) mx.add(w[h][i]);
    if constexpr (GLU) {
      if (!XQ && !YQ && !(live && c < a.C)) continue;
      const F<V> gate = unpack<T, V>(w[0][i]), val = unpack<T, V>(w[1][i]);
      F<V> v;
#pragma unroll
      for (int e = 0; e < V; ++e) v.v[e] = act<T>(gate.v[e], a.act) * val.v[e];
      if constexpr (YQ)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y[i][e] = v.v[e];
          my.m[e] = max32(my.m[e], __float_as_uint(v.v[e]));
        }
      if (a.y && live && c < a.C && DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) store_stream((T*)a.y + y0 + c * a.P, packed<T, V>(v));
    }
  }
  if constexpr (NM > 0) {
    // the largest over all threads of the same pixels: by shuffles inside the warp, then over the warps
    for (int o = g.LX; o < 32; o *= 2) {
      if constexpr (XQ)
#pragma unroll
        for (int k = 0; k < MX::N; ++k) mx.join(__shfl_xor_sync(0xffffffffu, mx.m[k], o), k);
      if constexpr (YQ)
#pragma unroll
        for (int k = 0; k < MY::N; ++k) my.join(__shfl_xor_sync(0xffffffffu, my.m[k], o), k);
    }
    const int warps = blockDim.x / 32, warp = tid / 32, row = NM * g.LX;
    if (warps > 1) {
      if ((tid & 31) < g.LX) {
        uint32_t* d = sums + warp * row + lx;
        if constexpr (XQ)
#pragma unroll
          for (int k = 0; k < MX::N; ++k) d[k * g.LX] = mx.m[k];
        if constexpr (YQ)
#pragma unroll
          for (int k = 0; k < MY::N; ++k) d[(NM - MY::N + k) * g.LX] = my.m[k];
      }
      __syncthreads();
      for (int o = 0; o < warps; ++o) {
        const uint32_t* d = sums + o * row + lx;
        if constexpr (XQ)
#pragma unroll
          for (int k = 0; k < MX::N; ++k) mx.join(d[k * g.LX], k);
        if constexpr (YQ)
#pragma unroll
          for (int k = 0; k < MY::N; ++k) my.join(d[(NM - MY::N + k) * g.LX], k);
      }
    }
  }
  if (!live) return;
  if constexpr (XQ) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const Quantizer z(mx.value(e));
      if (j0 == 0) a.xscale[b * a.P + p + e] = z.scale;
#pragma unroll
      for (int i = 0; i < J; ++i)
#pragma unroll
        for (int h = 0; h < G; ++h) {
          // the value's place takes its integer
          T v[V];
          memcpy(v, &w[h][i], sizeof(R));
          const uint32_t n = quantize<T>(to_f32(v[e]), z);
          if constexpr (sizeof(T) == 4) {
            uint32_t u[V];
            memcpy(u, &w[h][i], sizeof(R));
            u[e] = n;
            memcpy(&w[h][i], u, sizeof(R));
          } else {
            uint16_t u[V];
            memcpy(u, &w[h][i], sizeof(R));
            u[e] = (uint16_t)n;
            memcpy(&w[h][i], u, sizeof(R));
          }
        }
    }
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int c = j0 + i * g.NL;
      if (c < a.C && DISCO_IN_BOUNDS(b < a.B && p + V <= a.P))
#pragma unroll
        for (int h = 0; h < G; ++h) {
          int8_t* d = a.xq + G * y0 - (G - 1) * p + h * half + c * a.P;
          uint32_t r[V];
          if constexpr (sizeof(T) == 4) {
            memcpy(r, &w[h][i], sizeof(R));
          } else {
            uint16_t u[V];
            memcpy(u, &w[h][i], sizeof(R));
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = u[e];
          }
          store_bytes<V>(d, r);
        }
    }
  }
  if constexpr (YQ) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const Quantizer z(my.value(e));
      if (j0 == 0) a.scale[b * a.P + p + e] = z.scale;
#pragma unroll
      for (int i = 0; i < J; ++i) y[i][e] = __uint_as_float(quantize_near(y[i][e], z));
    }
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int c = j0 + i * g.NL;
      if (c < a.C && DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) {
        uint32_t r[V];
#pragma unroll
        for (int e = 0; e < V; ++e) r[e] = __float_as_uint(y[i][e]);
        store_bytes<V>(a.q + y0 + c * a.P, r);
      }
    }
  }
}

// Rows: `TR` threads (whole warps) take one token each, blockDim.x / TR tokens a CTA.
template <typename T, int V, int J, bool GLU, bool XQ, bool YQ>
__global__ void __launch_bounds__(kTokenThreads) tokens_rows_kernel(const TokenArgs a, const int TR) {
  constexpr int G = GLU ? 2 : 1;
  using R = Raw<T, V>;
  __shared__ float part[2][kTokenThreads / 32];
  const int tid = threadIdx.x, tr = tid % TR;
  const long long b = (long long)blockIdx.x * (blockDim.x / TR) + tid / TR;
  const bool live = b < a.B;
  const T* x = (const T*)a.x + b * G * a.C;
  const long long y0 = b * a.C;
  R w[G][J];
  float y[YQ ? J : 1][V];
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int c = (tr + i * TR) * V;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      memset(&w[h][i], 0, sizeof(R));
      if (live && c < a.C && DISCO_IN_BOUNDS(c + V <= a.C)) w[h][i] = load_stream<R>(x + h * a.C + c);
    }
  }
  Mag<T, V> mx;
  float my = 0.0f;
  mx.clear();
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int c = (tr + i * TR) * V;
    if constexpr (XQ)
#pragma unroll
      for (int h = 0; h < G; ++h) mx.add(w[h][i]);
    if constexpr (GLU) {
      const F<V> gate = unpack<T, V>(w[0][i]), val = unpack<T, V>(w[1][i]);
      F<V> v;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        v.v[e] = act<T>(gate.v[e], a.act) * val.v[e];
        if constexpr (YQ) {
          y[i][e] = v.v[e];
          my = __uint_as_float(max32(__float_as_uint(my), __float_as_uint(v.v[e])));
        }
      }
      if (a.y && live && c < a.C && DISCO_IN_BOUNDS(c + V <= a.C)) store_stream((T*)a.y + y0 + c, packed<T, V>(v));
    }
  }
  // the largest over the token's threads
  float m[2] = {XQ ? mx.all() : 0.0f, my};
  if constexpr (XQ || YQ) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k == 0 ? XQ : YQ)
        m[k] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m[k])));
    if (TR > 32) {
      if ((tid & 31) == 0) part[0][tid / 32] = m[0], part[1][tid / 32] = m[1];
      __syncthreads();
      for (int o = tid / TR * (TR / 32), n = TR / 32; n > 0; ++o, --n)
#pragma unroll
        for (int k = 0; k < 2; ++k) m[k] = __uint_as_float(max(__float_as_uint(m[k]), __float_as_uint(part[k][o])));
    }
  }
  if (!live) return;
  if constexpr (XQ) {
    const Quantizer z(m[0]);
    if (tr == 0) a.xscale[b] = z.scale;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int c = (tr + i * TR) * V;
      if (c < a.C && DISCO_IN_BOUNDS(c + V <= a.C))
#pragma unroll
        for (int h = 0; h < G; ++h) {
          const F<V> f = unpack<T, V>(w[h][i]);
          uint32_t r[V];
#pragma unroll
          for (int e = 0; e < V; ++e) r[e] = quantize<T>(f.v[e], z);
          store_bytes<V>(a.xq + G * y0 + h * a.C + c, r);
        }
    }
  }
  if constexpr (YQ) {
    const Quantizer z(m[1]);
    if (tr == 0) a.scale[b] = z.scale;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int c = (tr + i * TR) * V;
      if (c < a.C && DISCO_IN_BOUNDS(c + V <= a.C)) {
        uint32_t r[V];
#pragma unroll
        for (int e = 0; e < V; ++e) r[e] = quantize_near(y[i][e], z);
        store_bytes<V>(a.q + y0 + c, r);
      }
    }
  }
}

// ---- grids: tiles of pixels in a ring of shared memory ----------------------

// Persistent CTAs of NT threads take tiles of LX words of pixels by all channels.  A
// thread copies its own words of the tiles ahead with cp.async, so the loads of `depth`
// tiles are in flight while one is worked on, and no barrier orders the copies; it reads its
// words twice (magnitudes, rounding).  y waits between the two in the words of its gate and value.
struct RingCut {
  int NT, LX, nj, depth;        // nj: words of a thread in a tile, of each half
  long long per_sample, tiles;
};
constexpr int kRingMax = 512;

// Reciprocal and magnitude of V tokens, as the words of a row of shared memory.
// Tokens of ordinary magnitudes need no power of two (Quantizer's f is 1); of zeros
// any magnitude gives 0.  A tile with any other token rounds one value at a time.
__device__ __forceinline__ bool ordinary(float amax) { return amax == 0.0f || (amax >= 1e-20f && amax <= 1e30f); }

// q of a word of V inputs of V tokens: quantize<T>, two values to an instruction
template <typename T, int V>
__device__ __forceinline__ void quantize_word(uint32_t (&r)[V], const F<V>& x, const F<V>& inv, const F<V>& minus_a, bool plain) {
  if (plain && sizeof(T) == 2) {
    const F<V> kx = norm::mul(norm::fill<V>(kQMax), x);
    F<V> t = norm::mul(kx, inv);
    t = norm::fma(norm::fma(t, minus_a, kx), inv, t);
    t = norm::add(t, norm::fill<V>(kRound));
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = __float_as_uint(t.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      Quantizer z(1.0f);
      if (plain) z.k = kQMax, z.b = -minus_a.v[e], z.inv = inv.v[e];
      else z = Quantizer(-minus_a.v[e]);
      r[e] = quantize<T>(x.v[e], z);
    }
  }
}

template <typename T, bool GLU, bool XQ, bool YQ>
__global__ void __launch_bounds__(kRingMax) tokens_ring_kernel(const TokenArgs a, const RingCut g) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES, G = GLU ? 2 : 1, kSum = (XQ ? ES : 0) + (YQ ? 4 : 0);
  using R = Raw<T, V>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lx = tid & (g.LX - 1), j0 = tid / g.LX, NL = g.NT / g.LX;
  const int warps = g.NT / 32, warp = tid / 32;
  const int slot_words = G * g.nj * g.NT;
  uint4* ring = reinterpret_cast<uint4*>(smem) + tid;
  float* scratch = reinterpret_cast<float*>(smem + (size_t)g.depth * slot_words * 16);  // of each warp: 1/a, -a of x, 127/a of y
  uint8_t* sums = reinterpret_cast<uint8_t*>(scratch + warps * ((XQ ? 2 : 0) + (YQ ? 1 : 0)) * g.LX * V);  // [2]: [warps][pixels] of x, of y
  const long long half = a.C * a.P;
  auto place = [&](long long t, long long* b, long long* p) {
    *b = g.tiles <= 0xffffffffLL ? (long long)((uint32_t)t / (uint32_t)g.per_sample) : t / g.per_sample;
    *p = (t - *b * g.per_sample) * (g.LX * V) + lx * V;
  };
  auto fetch = [&](long long t, int slot) {
    if (t < g.tiles) {
      long long b, p;
      place(t, &b, &p);
      if (p < a.P) {
        const T* x = (const T*)a.x + b * G * half + p;
        uint4* d = ring + slot * slot_words;
        for (int i = 0; i < g.nj; ++i) {
          const int c = j0 + i * NL;
          if (c < a.C && DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) {
#pragma unroll
            for (int h = 0; h < G; ++h) norm::copy_async(d + (i * G + h) * g.NT, x + h * half + c * a.P);
          }
        }
      }
    }
    norm::copy_commit();
  };
  for (int d = 0; d < g.depth - 1; ++d) fetch(blockIdx.x + (long long)d * gridDim.x, d);
  int n = 0;
  for (long long t = blockIdx.x; t < g.tiles; t += gridDim.x, ++n) {
    fetch(t + (long long)(g.depth - 1) * gridDim.x, (n + g.depth - 1) % g.depth);
    if (g.depth == 3) norm::copy_wait<2>();
    else norm::copy_wait<1>();
    long long b, p;
    place(t, &b, &p);
    const bool live = p < a.P;
    const long long y0 = b * half + p;
    uint4* w = ring + (n % g.depth) * slot_words;
    Mag<T, V> mx;
    uint32_t my[V];
    mx.clear();
#pragma unroll
    for (int e = 0; e < V; ++e) my[e] = 0;
    const int nj = live ? (a.C - j0 + NL - 1) / NL : 0;
#pragma unroll 2
    for (int i = 0; i < nj; ++i) {
      uint4* s = w + i * G * g.NT;
      const uint4 w0 = s[0];
      if constexpr (XQ) mx.add(w0);
      if constexpr (GLU) {
        const uint4 w1 = s[g.NT];
        if constexpr (XQ) mx.add(w1);
        R r0, r1;
        memcpy(&r0, &w0, 16);
        memcpy(&r1, &w1, 16);
        const F<V> gate = unpack<T, V>(r0), val = unpack<T, V>(r1);
        F<V> v;
#pragma unroll
        for (int e = 0; e < V; ++e) v.v[e] = act<T>(gate.v[e], a.act) * val.v[e];
        if constexpr (YQ) {
#pragma unroll
          for (int e = 0; e < V; ++e) my[e] = max32(my[e], __float_as_uint(v.v[e]));
          if constexpr (!XQ) {  // y over its gate and value
            s[0] = *reinterpret_cast<const uint4*>(v.v);
            if constexpr (V == 8) s[g.NT] = *reinterpret_cast<const uint4*>(v.v + 4);
          }
        }
        if (a.y && DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) store_stream((T*)a.y + y0 + (j0 + i * NL) * a.P, packed<T, V>(v));
      }
    }
    const int TP = g.LX * V;
    float* own = scratch + warp * ((XQ ? 2 : 0) + (YQ ? 1 : 0)) * TP;
    bool plain = true;
    if constexpr (XQ || YQ) {
      for (int o = g.LX; o < 32; o *= 2) {
        if constexpr (XQ)
#pragma unroll
          for (int k = 0; k < Mag<T, V>::N; ++k) mx.join(__shfl_xor_sync(0xffffffffu, mx.m[k], o), k);
        if constexpr (YQ)
#pragma unroll
          for (int k = 0; k < V; ++k) my[k] = max(my[k], __shfl_xor_sync(0xffffffffu, my[k], o));
      }
      // rows of the tile's pixels, one for each warp; two sets of them: one barrier a tile
      uint8_t* part = sums + (n & 1) * warps * TP * kSum;
      if ((tid & 31) < g.LX) {
        if constexpr (XQ) memcpy(part + (warp * TP + lx * V) * ES, mx.m, V * ES);
        if constexpr (YQ) memcpy(part + warps * TP * (XQ ? ES : 0) + (warp * TP + lx * V) * 4, my, V * 4);
      }
      __syncthreads();
      // each warp joins them for itself, a pixel to a lane
      for (int e = tid & 31; e < TP; e += 32) {
        const long long at = b * a.P + p - lx * V + e;
        const bool in = p - lx * V + e < a.P;
        if constexpr (XQ) {
          float amax;
          if constexpr (ES == 2) {
            uint32_t m = 0;
            for (int o = 0; o < warps; ++o) m = max(m, (uint32_t)reinterpret_cast<const uint16_t*>(part)[o * TP + e]);
            const uint16_t h = (uint16_t)m;
            T v;
            memcpy(&v, &h, 2);
            amax = to_f32(v);
          } else {
            uint32_t m = 0;
            for (int o = 0; o < warps; ++o) m = max(m, reinterpret_cast<const uint32_t*>(part)[o * TP + e]);
            amax = __uint_as_float(m);
          }
          plain = plain && ordinary(amax);
          if (warp == 0 && in) a.xscale[at] = Quantizer(amax).scale;
          own[e] = __frcp_rn(amax == 0.0f ? 1.0f : amax);
          own[TP + e] = amax == 0.0f ? -1.0f : -amax;
        }
        if constexpr (YQ) {
          const uint32_t* q = reinterpret_cast<const uint32_t*>(part + warps * TP * (XQ ? ES : 0));
          uint32_t m = 0;
          for (int o = 0; o < warps; ++o) m = max(m, q[o * TP + e]);
          const Quantizer z(__uint_as_float(m));
          if (warp == 0 && in) a.scale[at] = z.scale;
          // a token with an infinity or a NaN: 0, and values that are NaN times it are cleared below
          own[(XQ ? 2 * TP : 0) + e] = z.scale < __int_as_float(0x7f800000) ? z.k * z.inv : 0.0f;
          plain = plain && z.scale < __int_as_float(0x7f800000);
        }
      }
      plain = __all_sync(0xffffffffu, plain);
      __syncwarp();
    }
    if (live) {
      if constexpr (XQ) {
        const F<V> inv = norm::load_row<V>(own + lx * V), minus_a = norm::load_row<V>(own + TP + lx * V);
        int8_t* d = a.xq + G * b * half + p + j0 * a.P;
#pragma unroll 2
        for (int i = 0; i < nj; ++i, d += NL * a.P)
#pragma unroll
          for (int h = 0; h < G; ++h) {
            R r0;
            memcpy(&r0, &w[(i * G + h) * g.NT], 16);
            uint32_t r[V];
            quantize_word<T, V>(r, unpack<T, V>(r0), inv, minus_a, plain);
            if (DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) store_bytes<V>(d + h * half, r);
          }
      }
      if constexpr (YQ) {
        const F<V> f = norm::load_row<V>(own + (XQ ? 2 * TP : 0) + lx * V);
        int8_t* d = a.q + y0 + j0 * a.P;
#pragma unroll 2
        for (int i = 0; i < nj; ++i, d += NL * a.P) {
          uint4* s = w + i * G * g.NT;
          F<V> v;
          if constexpr (!XQ) {
            *reinterpret_cast<uint4*>(v.v) = s[0];
            if constexpr (V == 8) *reinterpret_cast<uint4*>(v.v + 4) = s[g.NT];
          } else {
            R r0, r1;
            memcpy(&r0, &s[0], 16);
            memcpy(&r1, &s[g.NT], 16);
            const F<V> gate = unpack<T, V>(r0), val = unpack<T, V>(r1);
#pragma unroll
            for (int e = 0; e < V; ++e) v.v[e] = act<T>(gate.v[e], a.act) * val.v[e];
          }
          v = norm::mul(v, f);
          if (!plain)
#pragma unroll
            for (int e = 0; e < V; ++e) v.v[e] = fabsf(v.v[e]) < 128.0f ? v.v[e] : 0.0f;
          v = norm::add(v, norm::fill<V>(kRound));
          uint32_t r[V];
#pragma unroll
          for (int e = 0; e < V; ++e) r[e] = __float_as_uint(v.v[e]);
          if (DISCO_IN_BOUNDS(b < a.B && p + V <= a.P)) store_bytes<V>(d, r);
        }
      }
    }
    __syncwarp();  // `own` is read
  }
}

template <typename T, bool GLU, bool XQ, bool YQ>
int tokens_ring(const TokenArgs& a, cudaStream_t st) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES, G = GLU ? 2 : 1, kSum = (XQ ? ES : 0) + (YQ ? 4 : 0), kOwn = (XQ ? 2 : 0) + (YQ ? 1 : 0);
  RingCut g;
  size_t smem = 0;
  // 128 bytes of a row to a tile, three tiles deep, while they fit
  static const int shapes[][2] = {{8, 3}, {8, 2}, {4, 2}, {2, 2}};
  bool fits = false;
  for (const auto& s : shapes) {
    g.LX = s[0], g.depth = s[1];
    while (g.LX > 2 && (long long)g.LX / 2 * V >= a.P) g.LX /= 2;
    // few channels: more pixels to a tile, over which what a thread does once a tile is spread
    while (g.LX < 32 && a.C * g.LX < 1024 && g.LX * V < a.P) g.LX *= 2;
    // about 512 threads to an SM, whose shared memory holds so many rings
    const int rings = (int)max(1LL, (long long)(norm::kMaxSmem / ((size_t)g.depth * G * a.C * g.LX * 16 + 4096)));
    g.NT = kRingMax;
    while (g.NT > 128 && (g.NT * rings > 640 || a.C * g.LX < g.NT)) g.NT /= 2;
    g.nj = (a.C + g.NT / g.LX - 1) / (g.NT / g.LX);
    smem = (size_t)g.depth * G * g.nj * g.NT * 16 + (size_t)(g.NT / 32) * g.LX * V * (4 * kOwn + 2 * kSum);
    if ((fits = smem <= norm::kMaxSmem)) break;
  }
  if (!fits) return DISCO_ERR_UNSUPPORTED;
  g.per_sample = (a.P + g.LX * V - 1) / (g.LX * V);
  g.tiles = g.per_sample * a.B;
  auto kern = tokens_ring_kernel<T, GLU, XQ, YQ>;
  // one limit for all calls: host threads share it
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)norm::kMaxSmem) != cudaSuccess)
    return check_launch("tokens_ring_kernel attribute");
  const int ctas = (int)min((size_t)(1024 / g.NT), (norm::kMaxSmem + 1024) / (smem + 1024));
  kern<<<(int)min(g.tiles, (long long)kSMs * max(1, ctas)), g.NT, smem, st>>>(a, g);
  return check_launch("tokens_ring_kernel");
}

// Launches the kernels above; DISCO_ERR_UNSUPPORTED, without launching, for tokens
// that no CTA holds.
template <typename T, int V, int J, bool GLU, bool XQ, bool YQ>
int tokens_held(const TokenArgs& a, cudaStream_t st) {
  constexpr int NM = (XQ ? Mag<T, V>::N : 0) + (YQ ? Mag<float, V>::N : 0);
  if (a.P == 1) {
    const int words = (a.C + V - 1) / V;
    int TR = 32;
    while (TR < kTokenThreads && TR * J < words) TR *= 2;
    if (TR * J < words) return DISCO_ERR_UNSUPPORTED;
    const int rows = max(1, 128 / TR);  // of a CTA
    tokens_rows_kernel<T, V, J, GLU, XQ, YQ><<<(a.B + rows - 1) / rows, TR * rows, 0, st>>>(a, TR);
    return check_launch("tokens_rows_kernel");
  }
  TokenCut g;
  // 128 bytes of a row to a tile, less where the channels need the threads or there are few pixels
  g.LX = V > 1 ? 8 : 32;
  g.NL = (a.C + J - 1) / J;
  while (g.LX > 1 && (long long)g.LX * g.NL > kTokenThreads) g.LX /= 2;
  while (g.LX > 1 && (long long)g.LX / 2 * V >= a.P) g.LX /= 2;
  if ((long long)g.LX * g.NL > kTokenThreads) return DISCO_ERR_UNSUPPORTED;
  const int threads = (g.LX * g.NL + 31) / 32 * 32;
  g.TP = g.LX * V;
  g.per_sample = (a.P + g.TP - 1) / g.TP;
  const long long tiles = g.per_sample * a.B;
  if (tiles > 0x7fffffffLL) return DISCO_ERR_UNSUPPORTED;
  tokens_tile_kernel<T, V, J, GLU, XQ, YQ><<<(unsigned)tiles, threads, (size_t)threads / 32 * NM * g.LX * 4, st>>>(a, g);
  return check_launch("tokens_tile_kernel");
}

}  // namespace i8
}  // namespace disco
