// disco_tokens.cuh -- the kernels that work token by token, each token's values held
// in registers between the join of the largest magnitude and the rounding
// (disco_quant_i8, disco_glu).  Not part of the ABI.
//
// A token's C values are dealt over the threads of one CTA.
//   tokens_tile_kernel   grids, V pixels (16 bytes) to a word: words in shared memory.  Where V does not
//                        divide P (ODD), aligned words are shifted on the way in and out
//   tokens_skew_kernel   quantisation where V does not divide P: aligned words as they are, which
//                        are not pixels ([1,512,259199] 118 us; shifted 192)
//   tokens_rows_kernel   rows (P = 1), J words of neighbouring channels to a thread, in registers
//   tokens_pixel_kernel  grids of more channels than the tiles hold: one pixel of J channels to a thread
// Bound by HBM where a thread has 16 to 32 words and three CTAs or more share an SM: one
// loads while another rounds.  Measured (GB300, bf16): quantisation of [1,512,360x720]
// 73 us, 5.4 TB/s (the same tile three deep in one CTA of 512 threads 117); of 16384 rows
// of 2048 18 us, 5.5 TB/s; gated activation of 2 x 128 channels on 361x720 to 16 bits 72 us, 5.5
// TB/s, to 8 bits 73, with the 8-bit input 102, on 361x719 144, 154 and 221.
#pragma once

#include <type_traits>

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
  int LX, NL;           // threads along pixels, along channels
  long long per_sample; // tiles of a sample
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

// the low bytes of V words
template <int V>
__device__ __forceinline__ typename Word<V>::type bytes_word(const uint32_t (&r)[V]) {
  typename Word<V>::type o;
  if constexpr (V == 1) {
    o = (uint8_t)r[0];
  } else {
    uint32_t w[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) w[i] = bytes4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
    memcpy(&o, w, V);
  }
  return o;
}
template <int V>
__device__ __forceinline__ void store_bytes(int8_t* p, const uint32_t (&r)[V]) {
  store_stream(p, bytes_word<V>(r));
}

// GLU: x holds gates and values, 2 C channels; y = act(gate) value.  XQ: the 8-bit
// form of x; YQ: that of y.
template <typename T, int J, bool GLU, bool XQ, bool YQ>
__global__ void __launch_bounds__(kTokenThreads) tokens_pixel_kernel(const TokenArgs a, const TokenCut g) {
  constexpr int G = GLU ? 2 : 1, NM = (XQ ? 1 : 0) + (YQ ? 1 : 0);
  extern __shared__ uint32_t part[];  // [warps][NM][LX]
  const int tid = threadIdx.x, lx = tid & (g.LX - 1), j0 = tid / g.LX;
  const long long t = blockIdx.x, b = t / g.per_sample, p = (t - b * g.per_sample) * g.LX + lx;
  const bool live = p < a.P && DISCO_IN_BOUNDS(b < a.B);
  const long long half = a.C * a.P, y0 = b * half + p, x0 = b * G * half + p;
  float w[G][J], y[YQ ? J : 1];
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int c = j0 + i * g.NL;
#pragma unroll
    for (int h = 0; h < G; ++h) w[h][i] = live && c < a.C ? to_f32(((const T*)a.x)[x0 + h * half + c * a.P]) : 0.0f;
  }
  uint32_t m[2] = {0, 0};  // magnitudes of x, of y
#pragma unroll
  for (int i = 0; i < J; ++i) {
    const int c = j0 + i * g.NL;
    if constexpr (XQ)
#pragma unroll
      for (int h = 0; h < G; ++h) m[0] = max32(m[0], __float_as_uint(w[h][i]));
    if constexpr (GLU) {
      const float v = gated<T, 1>({{w[0][i]}}, {{w[1][i]}}, a.act).v[0];
      if constexpr (YQ) {
        y[i] = v;
        m[1] = __float_as_uint(max_abs(__uint_as_float(m[1]), v));
      }
      if (a.y && live && c < a.C) ((T*)a.y)[y0 + c * a.P] = from_f32<T>(v);
    }
  }
  if constexpr (NM > 0) {
    // the largest over all threads of the same pixel: by shuffles inside the warp, then over the warps
    for (int o = g.LX; o < 32; o *= 2)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (k ? YQ : XQ) m[k] = max(m[k], __shfl_xor_sync(0xffffffffu, m[k], o));
    const int warps = blockDim.x / 32;
    if (warps > 1) {
      if ((tid & 31) < g.LX)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k ? YQ : XQ) part[(tid / 32 * NM + (k && XQ)) * g.LX + lx] = m[k];
      __syncthreads();
      for (int o = 0; o < warps; ++o)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (k ? YQ : XQ) m[k] = max(m[k], part[(o * NM + (k && XQ)) * g.LX + lx]);
    }
  }
  if (!live) return;
  if constexpr (XQ) {
    const Quantizer z(__uint_as_float(m[0]));
    if (j0 == 0) a.xscale[b * a.P + p] = z.scale;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int c = j0 + i * g.NL;
      if (c < a.C)
#pragma unroll
        for (int h = 0; h < G; ++h) a.xq[x0 + h * half + c * a.P] = (int8_t)quantize<T>(w[h][i], z);
    }
  }
  if constexpr (YQ) {
    const Quantizer z(__uint_as_float(m[1]));
    if (j0 == 0) a.scale[b * a.P + p] = z.scale;
#pragma unroll
    for (int i = 0; i < J; ++i) {
      const int c = j0 + i * g.NL;
      if (c < a.C) a.q[y0 + c * a.P] = (int8_t)quantize_y<T>(y[i], z);
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
      const F<V> v = gated<T, V>(gate, val, a.act);
      if constexpr (YQ)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          y[i][e] = v.v[e];
          my = max_abs(my, v.v[e]);
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
        for (int e = 0; e < V; ++e) r[e] = quantize_y<T>(y[i][e], z);
        store_bytes<V>(a.q + y0 + c, r);
      }
    }
  }
}

// ---- grids: tiles of pixels in shared memory --------------------------------

// Persistent CTAs of NT threads take tiles of LX words of pixels by all channels.  A
// thread copies its own words of a tile with cp.async and reads them twice (magnitudes,
// rounding).  y waits between the two in the words of its gate and value.
struct TileCut {
  int NT, LX, nj;  // nj: words of a thread in a tile, of each half
  int roomy = 0;   // sample b < roomy - 1 is followed by two words of x, so its rows' last words end inside x
  long long per_sample, tiles;
};
constexpr int kTileThreads = 512;

// Reciprocal and magnitude of V tokens, as the words of a row of shared memory.
// Tokens of ordinary magnitudes need no power of two (Quantizer's f is 1); of zeros
// any magnitude gives 0.  A tile with any other token rounds one value at a time.
__device__ __forceinline__ bool ordinary(float amax) { return amax == 0.0f || (amax >= 1e-20f && amax <= 1e30f); }

// q of a word of V inputs of V tokens: quantize<T>, two values to an instruction
template <typename T, int V, bool PLAIN>
__device__ __forceinline__ void quantize_word(uint32_t (&r)[V], const F<V>& x, const F<V>& inv, const F<V>& minus_a) {
  if constexpr (PLAIN && sizeof(T) == 2) {
    const F<V> kx = norm::mul(norm::fill<V>(kQMax), x);
    F<V> t = norm::mul(kx, inv);
    t = norm::fma(norm::fma(t, minus_a, kx), inv, t);
    t = norm::add(t, norm::fill<V>(kRound));
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = __float_as_uint(t.v[e]);
  } else {
    if constexpr (PLAIN) {  // fp32: one test for the word (quantize<float>)
      const F<V> t = norm::mul(norm::mul(norm::fill<V>(kQMax), x), inv), u = norm::add(t, norm::fill<V>(kRound));
      const F<V> d = norm::add(norm::add(u, norm::fill<V>(-kRound)), norm::mul(t, norm::fill<V>(-1.0f)));
      float far = 0.0f;  // from the integers
#pragma unroll
      for (int e = 0; e < V; ++e) {
        far = fmaxf(far, fabsf(d.v[e]));
        r[e] = __float_as_uint(u.v[e]);
      }
      if (far < 0.5f - 0x1p-14f) return;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) r[e] = quantize<T>(x.v[e], Quantizer(-minus_a.v[e]));
  }
}

// V elements from element k on (nv of them wanted, zeros behind) of a tensor of `total`.
template <typename T, int V>
__device__ __forceinline__ uint4 load_px(const T* x, long long k, int nv, long long total) {
  constexpr int ES = (int)sizeof(T);
  const int m = (int)k & (V - 1);
  auto word = [&](long long at) {
    if (at + V <= total) return load_stream<uint4>(x + at);
    T v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = at + e < total ? x[at + e] : from_f32<T>(0.0f);
    uint4 w;
    memcpy(&w, v, 16);
    return w;
  };
  uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
  if (nv > 0 && DISCO_IN_BOUNDS(k - m >= 0 && k + nv <= total)) {
    lo = word(k - m);
    if (m + nv > V) hi = word(k - m + V);
  }
  return shifted(lo, hi, m * ES, nv * ES);
}

// The V pixels of each of LX lanes to a row that starts at element k, m past a word: N
// pixels of the tile.  Lanes put together aligned words from their own and their neighbour's
// pixels; the V pixels in words that another tile shares go out one to a lane.  All
// lanes of the warp call it; `has`: the row is there.
template <int V, typename W>
__device__ __forceinline__ void store_px(void* base, long long k, W word, int lx, int LX, int N, bool has) {
  constexpr int NW = (int)sizeof(W) / 4, ES = (int)sizeof(W) / V;
  using E = typename Word<ES>::type;
  const int m = (int)k & (V - 1);
  uint32_t w[NW], u[2 * NW + 1];
  memcpy(w, &word, sizeof(W));
#pragma unroll
  for (int i = 0; i < NW; ++i) u[i] = __shfl_up_sync(0xffffffffu, w[i], 1, LX), u[NW + i] = w[i];
  u[2 * NW] = 0;
  E* d = (E*)base + k;
  if (N == LX * V) {
    const int off = (V - m) * ES;  // where the aligned word starts in the neighbour's bytes and these
    // by whole words, then by bytes
#pragma unroll
    for (int step = NW; step >= 1; step /= 2)
      if (off / 4 & step) {
#pragma unroll
        for (int i = 0; i + step < 2 * NW + 1; ++i) u[i] = u[i + step];
      }
    uint32_t o[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) o[i] = ES % 4 ? __funnelshift_r(u[i], u[i + 1], 8 * (off & 3)) : u[i];
    memcpy(&word, o, sizeof(W));
    if (has && (lx > 0 || m == 0)) store_stream(d - m + lx * V, word);
    const int e = lx & (V - 1), from = e < V - m ? 0 : LX - 1;
    uint32_t one = 0;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const uint32_t x = __shfl_sync(0xffffffffu, w[i], from, LX);
      one = e * ES / 4 == i ? x : one;
    }
    if (has && m > 0 && lx < V) d[from * V + e] = (E)(one >> (8 * (e * ES & 3)));
  } else if (has) {
    E v[V];
    memcpy(v, &word, sizeof(W));
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (lx * V + e < N) d[lx * V + e] = v[e];
  }
}

template <typename T, bool GLU, bool XQ, bool YQ, bool ODD>
__global__ void __launch_bounds__(kTileThreads) tokens_tile_kernel(const TokenArgs a, const TileCut g) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES, G = GLU ? 2 : 1, kOwnY = XQ ? 2 : 0, kOwn = kOwnY + (YQ ? 2 : 0);
  using R = Raw<T, V>;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lx = tid & (g.LX - 1), j0 = tid / g.LX, NL = g.NT / g.LX, NT = g.NT, TP = g.LX * V;
  const int warps = NT / 32, warp = tid / 32;
  uint4* w = reinterpret_cast<uint4*>(smem) + tid;
  float* own = reinterpret_cast<float*>(smem + (size_t)G * g.nj * NT * 16);  // of each pixel: 1/a, -a of x, a and 127/a of y
  uint8_t* sums = reinterpret_cast<uint8_t*>(own + kOwn * TP);  // [warps][pixels] of x, of y
  const int nj = j0 < a.C ? (a.C - j0 + NL - 1) / NL : 0;       // channels of this thread
  const long long P = a.P, half = a.C * P, step = NL * P, row0 = j0 * P;  // from one of its channels to the next; its first
  for (long long t = blockIdx.x; t < g.tiles; t += gridDim.x) {
    const long long b = g.tiles <= 0xffffffffLL ? (long long)((uint32_t)t / (uint32_t)g.per_sample) : t / g.per_sample;
    const long long pos = (t - b * g.per_sample) * TP, p = pos + lx * V, y0 = b * half + p;
    const int N = (int)min((long long)TP, P - pos);  // pixels of the tile
    const bool live = p < P && DISCO_IN_BOUNDS(b < a.B);
    const int n = live ? nj : 0;
    const int loops = ODD ? g.nj : n;  // stores off alignment are the whole warp's
    if constexpr (ODD) {
      const long long k0 = b * G * half + p + row0, total = (long long)a.B * G * half;
      const int nv = min(V, N - lx * V);
      if (b + 1 < g.roomy || pos + TP + V <= P) {
        // both words of every row end inside the tensor: no tests between the loads, eight of them in flight
        constexpr int U = 4 / G;
        for (int i0 = 0; i0 < n; i0 += U) {
          uint4 lo[U][G], hi[U][G];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < G; ++h) {
              const long long k = k0 + min(i0 + u, n - 1) * step + h * half;
              const T* x = (const T*)a.x + (k & ~(long long)(V - 1));
              if (DISCO_IN_BOUNDS(k >= 0 && (k & ~(long long)(V - 1)) + 2 * V <= total)) lo[u][h] = load_stream<uint4>(x), hi[u][h] = load_stream<uint4>(x + V);
            }
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < G; ++h)
              if (i0 + u < n) {
                const int m = (int)(k0 + (i0 + u) * step + h * half) & (V - 1);
                w[((i0 + u) * G + h) * NT] = shifted(lo[u][h], hi[u][h], m * ES, nv * ES);
              }
        }
      } else {
        for (int i = 0; i < n; ++i)
#pragma unroll
          for (int h = 0; h < G; ++h) w[(i * G + h) * NT] = load_px<T, V>((const T*)a.x, k0 + i * step + h * half, nv, total);
      }
    } else {
      const T* x = (const T*)a.x + b * G * half + p + row0;
      uint4* d = w;
#pragma unroll 4
      for (int i = 0; i < n; ++i, x += step, d += G * NT) {
        norm::copy_async(d, x);
        if constexpr (GLU) norm::copy_async(d + NT, x + half);
      }
      norm::copy_commit();
      norm::copy_wait<0>();
    }
    Mag<T, V> mx;
    uint32_t my[V];
    mx.clear();
#pragma unroll
    for (int e = 0; e < V; ++e) my[e] = 0;
    {
      uint4* s = w;
      long long yo = y0 - lx * V * ODD + row0;
      auto first = [&](auto kind) {  // the activation's kind is known in the loop
#pragma unroll 4
        for (int i = 0; i < loops; ++i, s += G * NT) {
          const bool has = !ODD || i < n;
          const uint4 zero = make_uint4(0, 0, 0, 0), w0 = has ? s[0] : zero;
          if constexpr (XQ) mx.add(w0);
          if constexpr (GLU) {
            const uint4 w1 = has ? s[NT] : zero;
            if constexpr (XQ) mx.add(w1);
            R r0, r1;
            memcpy(&r0, &w0, 16);
            memcpy(&r1, &w1, 16);
            const F<V> v = gated<T, V>(unpack<T, V>(r0), unpack<T, V>(r1), decltype(kind)::value);
            if constexpr (YQ) {
#pragma unroll
              for (int e = 0; e < V; ++e) my[e] = __float_as_uint(max_abs(__uint_as_float(my[e]), v.v[e]));
              if constexpr (!XQ) {  // y over its gate and value
                if (has) {
                  s[0] = *reinterpret_cast<const uint4*>(v.v);
                  if constexpr (V == 8) s[NT] = *reinterpret_cast<const uint4*>(v.v + 4);
                }
              }
            }
            if (a.y) {
              if constexpr (ODD) store_px<V>(a.y, yo, packed<T, V>(v), lx, g.LX, N, i < nj);
              else store_stream((T*)a.y + yo, packed<T, V>(v));
              yo += step;
            }
          }
        }
      };
      if (GLU && a.act == DISCO_GELU) first(std::integral_constant<int, DISCO_GELU>());
      else first(std::integral_constant<int, DISCO_SILU>());
    }
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
      // rows of the tile's pixels, one for each warp
      uint8_t* ysums = sums + (XQ ? warps * TP * ES : 0);
      if ((tid & 31) < g.LX) {
        if constexpr (XQ) memcpy(sums + (warp * TP + lx * V) * ES, mx.m, V * ES);
        if constexpr (YQ) memcpy(ysums + (warp * TP + lx * V) * 4, my, V * 4);
      }
      __syncthreads();
      // S neighbouring threads to a pixel join them
      const int S = g.NT > TP ? g.NT / TP : 1, sub = tid & (S - 1);
      for (int e = tid / S; e < TP; e += g.NT / S) {
        const long long at = b * a.P + p - lx * V + e;
        const bool first = sub == 0, in = first && p - lx * V + e < a.P;
        if constexpr (XQ) {
          uint32_t m = 0;
          for (int o = sub; o < warps; o += S)
            m = max(m, ES == 2 ? (uint32_t)reinterpret_cast<const uint16_t*>(sums)[o * TP + e] : reinterpret_cast<const uint32_t*>(sums)[o * TP + e]);
          for (int o = 1; o < S; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          float amax = __uint_as_float(m);
          if constexpr (ES == 2) {
            const uint16_t h = (uint16_t)m;
            T v;
            memcpy(&v, &h, 2);
            amax = to_f32(v);
          }
          plain = plain && ordinary(amax);
          if (in) a.xscale[at] = Quantizer(amax).scale;
          if (first) {
            own[e] = __frcp_rn(amax == 0.0f ? 1.0f : amax);
            own[TP + e] = amax == 0.0f ? -1.0f : -amax;
          }
        }
        if constexpr (YQ) {
          const uint32_t* q = reinterpret_cast<const uint32_t*>(ysums);
          uint32_t m = 0;
          for (int o = sub; o < warps; o += S) m = max(m, q[o * TP + e]);
          for (int o = 1; o < S; o *= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          const float amax = __uint_as_float(m);
          const Quantizer z(amax);
          if (in) a.scale[at] = z.scale;
          if (first) own[kOwnY * TP + e] = amax, own[(kOwnY + 1) * TP + e] = z.k * z.inv;
          plain = plain && ordinary(amax);
        }
      }
      plain = __syncthreads_and(plain);
    }
    if constexpr (XQ) {
      const F<V> inv = norm::load_row<V>(own + lx * V), minus_a = norm::load_row<V>(own + TP + lx * V);
      auto second = [&](auto is_plain) {
        const uint4* s = w;
        long long d = G * b * half + (ODD ? pos : p) + row0;
#pragma unroll 4
        for (int i = 0; i < loops; ++i, s += G * NT, d += step)
#pragma unroll
          for (int h = 0; h < G; ++h) {
            R r0;
            const uint4 w0 = !ODD || i < n ? s[h * NT] : make_uint4(0, 0, 0, 0);
            memcpy(&r0, &w0, 16);
            uint32_t r[V];
            quantize_word<T, V, decltype(is_plain)::value>(r, unpack<T, V>(r0), inv, minus_a);
            if constexpr (ODD) store_px<V>(a.xq, d + h * half, bytes_word<V>(r), lx, g.LX, N, i < nj);
            else store_bytes<V>(a.xq + d + h * half, r);
          }
      };
      if (plain) second(std::true_type());
      else second(std::false_type());
    }
    if constexpr (YQ) {
      const F<V> amax = norm::load_row<V>(own + kOwnY * TP + lx * V), f = norm::load_row<V>(own + (kOwnY + 1) * TP + lx * V);
      auto third = [&](auto is_plain, auto kind) {
        const uint4* s = w;
        long long d = b * half + (ODD ? pos : p) + row0;
#pragma unroll 4
        for (int i = 0; i < loops; ++i, s += G * NT, d += step) {
          F<V> v;
          const bool has = !ODD || i < n;
          const uint4 zero = make_uint4(0, 0, 0, 0), w0 = has ? s[0] : zero;
          [[maybe_unused]] const uint4 w1 = (XQ || V == 8) && has ? s[NT] : zero;
          if constexpr (!XQ) {
            *reinterpret_cast<uint4*>(v.v) = w0;
            if constexpr (V == 8) *reinterpret_cast<uint4*>(v.v + 4) = w1;
          } else {
            R r0, r1;
            memcpy(&r0, &w0, 16);
            memcpy(&r1, &w1, 16);
            v = gated<T, V>(unpack<T, V>(r0), unpack<T, V>(r1), decltype(kind)::value);
          }
          uint32_t r[V];
          if constexpr (decltype(is_plain)::value && ES == 2) {
            v = norm::add(norm::mul(v, f), norm::fill<V>(kRound));
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = __float_as_uint(v.v[e]);
          } else if constexpr (decltype(is_plain)::value) {
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = __float_as_uint(__fdiv_rn(__fmul_rn(kQMax, v.v[e]), amax.v[e] == 0.0f ? 1.0f : amax.v[e]) + kRound);
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) r[e] = quantize_y<T>(v.v[e], Quantizer(amax.v[e]));
          }
          if constexpr (ODD) store_px<V>(a.q, d, bytes_word<V>(r), lx, g.LX, N, i < nj);
          else store_bytes<V>(a.q + d, r);
        }
      };
      using Silu = std::integral_constant<int, DISCO_SILU>;
      using Gelu = std::integral_constant<int, DISCO_GELU>;
      if (XQ && a.act == DISCO_GELU) third(std::false_type(), Gelu());
      else if (plain) third(std::true_type(), Silu());
      else third(std::false_type(), Silu());
    }
  }
}

template <typename T, bool GLU, bool XQ, bool YQ, bool ODD>
int tokens_tiles(const TokenArgs& a, cudaStream_t st) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES, G = GLU ? 2 : 1, kSum = (XQ ? ES : 0) + (YQ ? 4 : 0), kOwn = (XQ ? 2 : 0) + (YQ ? 2 : 0);
  TileCut g;
  // 128 bytes of a row to a tile, more for few channels, less for many, so that three tiles share an SM
  g.LX = 8;
  while (g.LX < 32 && (long long)G * a.C * g.LX < 1024 && g.LX * V < a.P) g.LX *= 2;
  // (shifted words want V lanes side by side)
  while (g.LX > (ODD ? V : 2) && ((size_t)G * a.C * g.LX * 16 * 3 > norm::kMaxSmem - 12 * 1024 || (long long)g.LX / 2 * V >= a.P)) g.LX /= 2;
  const int share = (int)(norm::kMaxSmem / ((size_t)G * a.C * g.LX * 16 + 4096));
  g.NT = share >= 3 ? (G * a.C * g.LX <= 1024 ? 64 : 128) : share == 2 ? 256 : kTileThreads;
  g.nj = (a.C + g.NT / g.LX - 1) / (g.NT / g.LX);
  const size_t smem = (size_t)G * g.nj * g.NT * 16 + (size_t)g.LX * V * (4 * kOwn + g.NT / 32 * kSum);
  if (smem > norm::kMaxSmem) return DISCO_ERR_UNSUPPORTED;
  // Samples of one channel by two pixels are shorter.  Decided here: in the kernel it cost
  // registers (2 x 128 channels on 361x719 with the checkpoint 221 us, 257 then).
  g.roomy = (long long)G * a.C * a.P >= 2 * V ? a.B : 0;
  g.per_sample = (a.P + g.LX * V - 1) / (g.LX * V);
  g.tiles = g.per_sample * a.B;
  auto kern = tokens_tile_kernel<T, GLU, XQ, YQ, ODD>;
  // one limit for all calls: host threads share it
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)norm::kMaxSmem) != cudaSuccess)
    return check_launch("tokens_tile_kernel attribute");
  const int ctas = (int)min((size_t)(1024 / g.NT), (norm::kMaxSmem + 1024) / (smem + 1024));
  kern<<<(int)min(g.tiles, (long long)kSMs * max(1, ctas)), g.NT, smem, st>>>(a, g);
  return check_launch("tokens_tile_kernel");
}

// Quantisation of grids where V does not divide P: a row of pixels starts m = 0 .. V - 1
// elements past a word.  Words stay aligned, LX of them cover TP = (LX - 1) V pixels and
// parts of two neighbouring tiles'; a thread's channels are a multiple of V apart, so its rows
// have one skew, and only its magnitudes and factors are realigned, once a tile.
template <typename T>
__global__ void __launch_bounds__(256) tokens_skew_kernel(const TokenArgs a, const TileCut g) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES;
  using R = Raw<T, V>;
  using M = typename Word<ES>::type;
  extern __shared__ __align__(16) uint8_t smem[];
  const int tid = threadIdx.x, lx = tid & (g.LX - 1), j0 = tid / g.LX, NL = g.NT / g.LX, TP = (g.LX - 1) * V, row = TP + 2 * V;
  uint4* w = reinterpret_cast<uint4*>(smem) + tid;
  float* own = reinterpret_cast<float*>(smem + (size_t)g.nj * g.NT * 16);  // 1/a and -a of pixels -V .. TP + V
  M* sums = reinterpret_cast<M*>(own + 2 * row);                           // [NL][pixels -V .. TP + V]
  const int nj = j0 < a.C ? (a.C - j0 + NL - 1) / NL : 0;
  const long long P = a.P, step = NL * P, total = (long long)a.B * a.C * P;
  for (long long t = blockIdx.x; t < g.tiles; t += gridDim.x) {
    const long long b = g.tiles <= 0xffffffffLL ? (long long)((uint32_t)t / (uint32_t)g.per_sample) : t / g.per_sample;
    const long long pos = (t - b * g.per_sample) * TP, e0 = (b * a.C + j0) * P + pos;
    const int N = (int)min((long long)TP, P - pos), m = (int)e0 & (V - 1), px = lx * V - m;  // this thread's first pixel
    const int n = px < N ? nj : 0;
    const long long at = e0 + px;  // its first element
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const long long k = at + i * step;
      const int left = DISCO_IN_BOUNDS(k >= 0 && k < total) ? (int)min((long long)V, total - k) : 0;
      norm::copy_async(w + i * g.NT, (const T*)a.x + (left ? k : 0), left * ES);
    }
    norm::copy_commit();
    norm::copy_wait<0>();
    Mag<T, V> mx;
    mx.clear();
#pragma unroll 4
    for (int i = 0; i < n; ++i) mx.add(w[i * g.NT]);
    M part[V];
    memcpy(part, mx.m, sizeof(part));
#pragma unroll
    for (int e = 0; e < V; ++e) sums[j0 * row + V + px + e] = part[e];
    __syncthreads();
    bool plain = true;
    for (int e = tid; e < N; e += g.NT) {
      uint32_t u = 0;
      for (int o = 0; o < NL; ++o) u = max(u, (uint32_t)sums[o * row + V + e]);
      const M h = (M)u;
      T v;
      memcpy(&v, &h, ES);
      const float amax = to_f32(v);
      plain = plain && ordinary(amax);
      a.xscale[b * P + pos + e] = Quantizer(amax).scale;
      own[V + e] = __frcp_rn(amax == 0.0f ? 1.0f : amax);
      own[row + V + e] = amax == 0.0f ? -1.0f : -amax;
    }
    plain = __syncthreads_and(plain);
    F<V> inv, minus_a;
#pragma unroll
    for (int e = 0; e < V; ++e) inv.v[e] = own[V + px + e], minus_a.v[e] = own[row + V + px + e];
    auto second = [&](auto is_plain) {
      using W = typename Word<V>::type;
      long long k = e0 - m;  // the element where the row's word 0 starts
#pragma unroll 2
      for (int i = 0; i < g.nj; ++i, k += step) {
        W o = {};
        if (i < n) {
          R r0;
          const uint4 w0 = w[i * g.NT];
          memcpy(&r0, &w0, 16);
          uint32_t r[V];
          quantize_word<T, V, decltype(is_plain)::value>(r, unpack<T, V>(r0), inv, minus_a);
          o = bytes_word<V>(r);
        }
        norm::store_words<V>(a.xq + k, k, total, o, m, lx, g.LX, N, i < nj);  // all lanes
      }
    };
    if (plain) second(std::true_type());
    else second(std::false_type());
  }
}

template <typename T>
int tokens_skewed(const TokenArgs& a, cudaStream_t st) {
  constexpr int ES = (int)sizeof(T), V = 16 / ES;
  TileCut g;
  // 15 words of pixels to a tile while three tiles share an SM, else 7 (at 3, half of the words are shared with other tiles)
  g.LX = (size_t)a.C * 16 * 16 * 3 <= norm::kMaxSmem - 24 * 1024 && 7 * V < a.P ? 16 : 8;
  g.NT = (size_t)a.C * g.LX * 16 * 3 <= norm::kMaxSmem - 24 * 1024 ? 128 : 256;  // a multiple of 8 channels side by side
  const int TP = (g.LX - 1) * V, NL = g.NT / g.LX;
  g.nj = (a.C + NL - 1) / NL;
  const size_t smem = (size_t)g.nj * g.NT * 16 + (size_t)(TP + 2 * V) * (8 + NL * ES);
  if (smem > norm::kMaxSmem) return DISCO_ERR_UNSUPPORTED;
  g.per_sample = (a.P + TP - 1) / TP;
  g.tiles = g.per_sample * a.B;
  const int ctas = (int)max((size_t)1, min((size_t)(1024 / g.NT), (norm::kMaxSmem + 1024) / (smem + 1024)));
  return norm::launch(tokens_skew_kernel<T>, (int)min(g.tiles, (long long)kSMs * ctas), g.NT, 1, false, smem, norm::kMaxSmem, st,
                      "tokens_skew_kernel", a, g);
}

// Launches the kernels above; DISCO_ERR_UNSUPPORTED, without launching, for tokens
// that no CTA holds.
template <typename T, int V, int J, bool GLU, bool XQ, bool YQ>
int held_as(const TokenArgs& a, cudaStream_t st) {
  [[maybe_unused]] constexpr int NM = (XQ ? 1 : 0) + (YQ ? 1 : 0);
  if (a.P == 1) {
    const int words = (a.C + V - 1) / V;
    const int TR = ((words + J - 1) / J + 31) / 32 * 32;
    if (TR > kTokenThreads) return DISCO_ERR_UNSUPPORTED;
    const int rows = max(1, 128 / TR);  // of a CTA
    tokens_rows_kernel<T, V, J, GLU, XQ, YQ><<<(unsigned)(((long long)a.B + rows - 1) / rows), TR * rows, 0, st>>>(a, TR);
    return check_launch("tokens_rows_kernel");
  }
  if constexpr (V > 1) {
    return DISCO_ERR_UNSUPPORTED;
  } else {
    TokenCut g;
    // 32 pixels of a row to a tile, fewer where the channels need the threads or there are few pixels
    g.LX = 32;
    g.NL = (a.C + J - 1) / J;
    while (g.LX > 1 && (long long)g.LX * g.NL > kTokenThreads) g.LX /= 2;
    while (g.LX > 1 && g.LX / 2 >= a.P) g.LX /= 2;
    const int threads = (g.LX * g.NL + 31) / 32 * 32;
    g.per_sample = (a.P + g.LX - 1) / g.LX;
    const long long tiles = g.per_sample * a.B;
    if ((long long)g.LX * g.NL > kTokenThreads || tiles > 0x7fffffffLL) return DISCO_ERR_UNSUPPORTED;
    tokens_pixel_kernel<T, J, GLU, XQ, YQ><<<(unsigned)tiles, threads, (size_t)threads / 32 * NM * g.LX * 4, st>>>(a, g);
    return check_launch("tokens_pixel_kernel");
  }
}

// By the element type, for tokens that the kernels hold (DISCO_ERR_UNSUPPORTED else): grids
// whose P words divide, other grids, and rows or single pixels.  glu: gates and values.
int tokens_grid(const TokenArgs& a, bool glu, disco_dtype dtype, cudaStream_t st);
int tokens_grid_odd(const TokenArgs& a, bool glu, disco_dtype dtype, cudaStream_t st);
int tokens_held(const TokenArgs& a, bool glu, disco_dtype dtype, cudaStream_t st);

template <typename T, bool ODD>
int tiles_of(const TokenArgs& a, bool glu, cudaStream_t st) {
  if (!glu) {
    if constexpr (ODD) return tokens_skewed<T>(a, st);
    else return tokens_tiles<T, false, true, false, false>(a, st);
  }
  if (a.xq && a.q) return tokens_tiles<T, true, true, true, ODD>(a, st);
  if (a.xq) return tokens_tiles<T, true, true, false, ODD>(a, st);
  if (a.q) return tokens_tiles<T, true, false, true, ODD>(a, st);
  return tokens_tiles<T, true, false, false, ODD>(a, st);
}

}  // namespace i8
}  // namespace disco
