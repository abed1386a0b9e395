// disco_norm_rows.cu -- the channel norm and its gradient on rows of features
// (P = 1: the C features of a row lie side by side).
//
// A team of LANES threads takes a row, each thread NWD aligned 16-byte words
// of it (word lane + i LANES).  Shared memory holds the words of the team's
// next rows as they arrive (thread-private cp.async, several rows ahead where a
// row is short).  Teams are parts of a warp, warps, or several warps of a CTA of
// kThreads threads; the latter meet at a named barrier.
//
// Where V (elements of a word) does not divide C, row b starts m = b C mod V
// elements past a word boundary.  m repeats every `period` rows, and a unit (a
// warp, or a team of several warps) only takes rows of one residue: a thread's
// words hold the same features in all its rows, so the gain and the sums of
// dweight stay in registers.  The first and last word of a row are partial.
//
// Measured (calls, GB300): [16384,2048] bf16, residual, h, q and scales in groups
// of 128: 42.6 us, 5.5 TB/s (82 % of the copy rate, DRAM 57 % busy, issue 53 %: the
// 8-bit form is bound by instructions); 2560 rows of 15507 features 55 us, 5.7 TB/s;
// 1600 rows of 24576 90 us, 3.5 TB/s (8 words to a thread: 128 registers, with
// spills); [12518,1693] with q, one group, 45 us, 4.2 TB/s (partial words).
// Gradient and the sum of dweight: [16384,2048] 45.1 us, 4.5 TB/s;
// [8599,6164] 133 us, 2.4 TB/s (issue 56 %, 16 warps to an SM: one row's join is
// waited for before the next row's sums begin).  16 rows of 512: a kernel of 5 us,
// the latency of a launch and one load.

#include "disco_norm.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_rows_bounds)

namespace norm {

namespace {

constexpr int kThreads = 512;

struct Rows {
  int LANES, NWD, NT;   // threads of a team, words of a thread, threads of a CTA
  int U;                // teams of a unit (a warp of small teams; else 1)
  int units;            // of the launch, a multiple of period
  int grid, period;
};

// A thread's place: its team's rows and its words' elements.  WHOLE: V divides
// C, every word is whole or past the row.
template <typename T, int NWD, bool WHOLE>
struct Place {
  static constexpr int V = 16 / (int)sizeof(T);
  int lane, team, LANES, B, C, m;  // team: of the CTA
  long long row, step, lead;       // first row; rows to the next one; first row of the unit (loops run by units)
  long long total;                 // elements of a tensor
  __device__ __forceinline__ Place(const Rows& g, int B_, int C_) : LANES(g.LANES), B(B_), C(C_), total((long long)B_ * C_) {
    lane = threadIdx.x & (LANES - 1);
    team = threadIdx.x / LANES;
    const int per_cta = LANES < 32 ? g.NT / 32 : g.NT / LANES;
    const int unit = blockIdx.x * per_cta + (LANES < 32 ? threadIdx.x / 32 : team);
    const int u = LANES < 32 ? (threadIdx.x & 31) / LANES : 0;
    const int rho = unit % g.period;
    const long long first = (long long)(unit / g.period) * g.U;
    row = rho + g.period * (first + u);
    lead = rho + g.period * first;
    step = (long long)g.U * g.units;
    m = WHOLE ? 0 : (int)((unsigned)(row * C) & (V - 1));
  }
  // Keeps the compiler from carrying every word's and element's tests on m
  // through the loop in registers.
  __device__ __forceinline__ void recompute() {
    if (!WHOLE) asm volatile("" : "+r"(m));
  }
  __device__ __forceinline__ int at(int i) const { return (lane + i * LANES) * V - m; }  // feature of word i's first element
  __device__ __forceinline__ bool any(int i) const { return at(i) < C; }
  __device__ __forceinline__ bool whole(int i) const { return WHOLE ? any(i) : at(i) >= 0 && at(i) + V <= C; }
  __device__ __forceinline__ bool in(int i, int e) const { return WHOLE ? any(i) : at(i) + e >= 0 && at(i) + e < C; }
  // element offset of word 0 of row r in the tensor
  __device__ __forceinline__ long long origin(long long r) const { return r * C + at(0); }
  // Elements from row r's first to the tensor's end, or more than the row's words
  // hold.  The words of the last row, and with rows shorter than a word those of
  // the rows before it, would end past the tensor.
  __device__ __forceinline__ int rest(long long r) const {
    return !WHOLE && r >= B - 1 - (V - 2) / C ? (int)(B - r) * C : C + V;
  }
  // a row whose origin is o, left = rest() of it
  __device__ __forceinline__ void fetch(const T* p, uint4* to, int NT, long long o, int left) const {
#pragma unroll
    for (int i = 0; i < NWD; ++i)
      if (any(i)) {
        const int bytes = WHOLE ? 16 : min((left - at(i)) * (int)sizeof(T), 16);
        const long long word = o + i * LANES * V;
        if (DISCO_IN_BOUNDS(word >= 0 && word + bytes / (int)sizeof(T) <= total)) copy_async(to + i * NT, p + word, bytes);
      }
  }
  // the elements of word i that are the row's; zeros in place of the others
  __device__ __forceinline__ F<V> own(F<V> v, int i) const {
    if (!WHOLE && !whole(i))
#pragma unroll
      for (int e = 0; e < V; ++e) v.v[e] = in(i, e) ? v.v[e] : 0.0f;
    return v;
  }
  template <typename W>
  __device__ __forceinline__ void write(void* p, long long o, int i, W w) const {
    constexpr int ES = (int)sizeof(W) / V;
    const long long word = o + i * LANES * V;
    char* d = (char*)p + word * ES;
    if (whole(i)) {
      if (DISCO_IN_BOUNDS(word >= 0 && word + V <= total)) store_stream(d, w);
    } else if (!WHOLE && any(i)) {
      const uint8_t* b = (const uint8_t*)&w;
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (in(i, e) && DISCO_IN_BOUNDS(word + e >= 0 && word + e < total)) {
          typename Word<ES>::type v;
          memcpy(&v, b + e * ES, ES);
          store_stream(d + e * ES, v);
        }
    }
  }
  __device__ __forceinline__ Raw<T, V> weight(const T* w, int i) const {
    T t[V];
#pragma unroll
    for (int e = 0; e < V; ++e) t[e] = w ? (in(i, e) ? w[at(i) + e] : from_f32<T>(0.0f)) : from_f32<T>(1.0f);
    Raw<T, V> r;
    memcpy(&r, t, sizeof(r));
    return r;
  }
  __device__ __forceinline__ void barrier() const {
    if (LANES <= 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(LANES) : "memory");
  }
  // N values over the team's threads; buf: this row's parity of two
  template <int N, typename Op>
  __device__ __forceinline__ void reduce(float (&v)[N], float (&buf)[N][kThreads / 32], Op op) const {
#pragma unroll
    for (int k = 16; k; k >>= 1)
      if (k < LANES)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = op(v[n], __shfl_xor_sync(0xffffffffu, v[n], k));
    if (LANES <= 32) return;
    const int w0 = team * (LANES / 32), nw = LANES / 32;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) buf[n][threadIdx.x / 32] = v[n];
    barrier();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = buf[n][w0];
      for (int k = 1; k < nw; ++k) v[n] = op(v[n], buf[n][w0 + k]);
    }
  }
};

// Rows in the ring of a thread: the forward keeps kAhead of them in flight while
// it holds one in registers; the gradient reads its row twice from the ring, so
// one of its kDepth is the current row (kDepth = 1: nothing ahead, the row is too long).
constexpr int ahead_of(int NWD) { return NWD >= 4 ? 1 : 4 / NWD; }
constexpr int depth_of(int NWD) { return NWD == 8 ? 1 : NWD >= 2 ? 2 : 4; }

template <int V>
__device__ __forceinline__ float across(const F<V>& f) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) s += f.v[e];
  return s;
}

// 1 / x for x >= kAmaxFloor to an ulp (the e4m3 values it scales have 4 bits); 0
// for an infinite x
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// How a group's maximum is found: its words are the row; are gw = G / V
// neighbouring lanes'; or by atomic maxima in shared memory (not WHOLE).
enum { kRow = 0, kLanes = 1, kAtomic = 2 };

template <typename T, int NWD, bool Q, bool WHOLE>
__global__ void __launch_bounds__(kThreads) norm_rows_kernel(const NormArgs a, const Rows g, const int qmode) {
  constexpr int V = 16 / (int)sizeof(T);
  using W = Raw<T, V>;
  extern __shared__ __align__(16) char smem[];
  __shared__ float buf[2][2][1][kThreads / 32];
  Place<T, NWD, WHOLE> P(g, a.B, a.C);
  const T *x = (const T*)a.x, *res = (const T*)a.res;
  constexpr int kAhead = ahead_of(NWD);
  const int words = g.NT * NWD;  // of one row of all teams
  uint4 *rx = (uint4*)smem + threadIdx.x, *rr = rx + kAhead * words;
  W wt[NWD];
#pragma unroll
  for (int i = 0; i < NWD; ++i) {
    wt[i] = P.weight((const T*)a.w, i);
    if (!P.any(i))  // words past the row: zeros, never copied over
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        rx[k * words + i * g.NT] = make_uint4(0, 0, 0, 0);
        if (res) rr[k * words + i * g.NT] = make_uint4(0, 0, 0, 0);
      }
  }
  uint32_t* gm = (uint32_t*)(smem + (size_t)kAhead * words * 16 * (res ? 2 : 1)) + (size_t)P.team * a.NG;  // kAtomic
  const long long step_o = P.step * a.C;
  auto fetch = [&](long long r, long long o, int slot) {
    if (r < a.B) {
      const int left = P.rest(r);
      P.fetch(x, rx + slot * words, g.NT, o, left);
      if (res) P.fetch(res, rr + slot * words, g.NT, o, left);
    }
    copy_commit();
  };
  long long o = P.origin(P.row);
  for (int k = 0; k < kAhead; ++k) fetch(P.row + k * P.step, o + k * step_o, k);
  int parity = 0, slot = 0;
  for (long long lead = P.lead, row = P.row; lead < a.B;
       lead += P.step, row += P.step, o += step_o, parity ^= 1, slot = slot + 1 == kAhead ? 0 : slot + 1) {
    P.recompute();
    const bool on = row < a.B;
    F<V> v[NWD], s = fill<V>(0.0f);
    copy_wait<kAhead - 1>();
#pragma unroll
    for (int i = 0; i < NWD; ++i) {
      v[i] = unpack<T, V>(rx[slot * words + i * g.NT]);
      if (res) v[i] = add(v[i], unpack<T, V>(rr[slot * words + i * g.NT]));
    }
    fetch(row + kAhead * P.step, o + kAhead * step_o, slot);
#pragma unroll
    for (int i = 0; i < NWD; ++i) {
      v[i] = P.own(v[i], i);
      s = fma(v[i], v[i], s);
    }
    if (a.h && on)
#pragma unroll
      for (int i = 0; i < NWD; ++i) P.write(a.h, o, i, packed<T, V>(v[i]));
    float sum[1] = {across(s)};
    P.reduce(sum, buf[0][parity], [](float p, float q) { return p + q; });
    const F<V> r = fill<V>(inverse_rms(sum[0], a.inv_C, a.eps));
#pragma unroll
    for (int i = 0; i < NWD; ++i) v[i] = mul(mul(v[i], r), unpack<T, V>(wt[i]));
    if (a.y && on)
#pragma unroll
      for (int i = 0; i < NWD; ++i) P.write(a.y, o, i, packed<T, V>(v[i]));

    if constexpr (Q) {
      if (!WHOLE && qmode == kAtomic) {
        for (int k = P.lane; k < a.NG; k += P.LANES) gm[k] = 0u;
        P.barrier();
#pragma unroll
        for (int i = 0; i < NWD; ++i)
          if (P.any(i)) {
            int c = max(P.at(i), 0), grp = c / a.G, end = (grp + 1) * a.G;
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (P.in(i, e)) {
                c = P.at(i) + e;
                if (c == end) {
                  atomicMax(gm + grp, __float_as_uint(top));
                  top = 0.0f, ++grp, end += a.G;
                }
                top = fmaxf(top, fabsf(v[i].v[e]));  // a NaN does not count
              }
            atomicMax(gm + grp, __float_as_uint(top));
          }
        P.barrier();
#pragma unroll
        for (int i = 0; i < NWD; ++i)
          if (P.any(i)) {
            int c = max(P.at(i), 0), grp = c / a.G, end = (grp + 1) * a.G;
            float inv = kE4m3Max / fmaxf(__uint_as_float(gm[grp]), kAmaxFloor);
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (P.in(i, e)) {
                if (P.at(i) + e == end) {
                  ++grp, end += a.G;
                  inv = kE4m3Max / fmaxf(__uint_as_float(gm[grp]), kAmaxFloor);
                }
                v[i].v[e] *= inv;
              }
            if (on) P.write(a.q, o, i, packed_e4m3<V>(v[i]));
          }
        if (on)
          for (int k = P.lane; k < a.NG; k += P.LANES)
            a.scale[row * a.NG + k] = fmaxf(__uint_as_float(gm[k]), kAmaxFloor) / kE4m3Max;
        P.barrier();
      } else {
        float top[NWD], all[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < NWD; ++i) {
          top[i] = kAmaxFloor;
#pragma unroll
          for (int e = 0; e < V; ++e) top[i] = fmaxf(top[i], fabsf(v[i].v[e]));  // a NaN does not count
          all[0] = fmaxf(all[0], top[i]);
        }
        if (qmode == kRow) {
          P.reduce(all, buf[1][parity], [](float p, float q) { return fmaxf(p, q); });
          if (on && P.lane == 0) a.scale[row] = all[0] / kE4m3Max;
        }
        if (qmode == kLanes) {
          const int gw = a.G / V;
#pragma unroll
          for (int k = 16; k; k >>= 1)
            if (k < gw)
#pragma unroll
              for (int i = 0; i < NWD; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], k));
          if (on && (P.lane & (gw - 1)) == 0) {
            float* to = a.scale + row * a.NG + P.lane / gw;
            const int next = P.LANES / gw;
#pragma unroll
            for (int i = 0; i < NWD; ++i)
              if (P.any(i)) to[i * next] = top[i] / kE4m3Max;
          }
        }
#pragma unroll
        for (int i = 0; i < NWD; ++i) {
          const float inv = kE4m3Max * reciprocal(qmode == kLanes ? top[i] : all[0]);
          if (on) P.write(a.q, o, i, packed_e4m3<V>(mul(v[i], fill<V>(inv))));
        }
      }
    }
  }
}

template <typename T, int NWD, bool WHOLE>
__global__ void __launch_bounds__(kThreads) norm_bwd_rows_kernel(const NormBwdArgs a, const Rows g) {
  constexpr int V = 16 / (int)sizeof(T);
  using W = Raw<T, V>;
  extern __shared__ __align__(16) char smem[];
  if (a.part) let_next_begin();
  __shared__ float buf[2][2][kThreads / 32];
  Place<T, NWD, WHOLE> P(g, a.B, a.C);
  const T *dy = (const T*)a.dy, *h = (const T*)a.h, *dh = (const T*)a.dh;
  constexpr int kDepth = depth_of(NWD);
  const int words = g.NT * NWD, streams = dh ? 3 : 2;  // words: of one row of all teams and one tensor
  uint4* ring = (uint4*)smem + threadIdx.x;            // [kDepth][dy, h, dh][NWD][NT]
  W wt[NWD];
  F<V> dw[NWD];
#pragma unroll
  for (int i = 0; i < NWD; ++i) {
    wt[i] = P.weight((const T*)a.w, i);
    dw[i] = fill<V>(0.0f);
    if (!P.any(i))  // words past the row: zeros, never copied over
#pragma unroll
      for (int k = 0; k < kDepth; ++k)
        for (int n = 0; n < streams; ++n) ring[(k * streams + n) * words + i * g.NT] = make_uint4(0, 0, 0, 0);
  }
  const long long step_o = P.step * a.C;
  auto fetch = [&](long long r, long long o, int slot) {
    if (r < a.B) {
      uint4* to = ring + slot * streams * words;
      const int left = P.rest(r);
      P.fetch(dy, to, g.NT, o, left);
      P.fetch(h, to + words, g.NT, o, left);
      if (dh) P.fetch(dh, to + 2 * words, g.NT, o, left);
    }
    copy_commit();
  };
  long long o = P.origin(P.row);
  for (int k = 0; k < kDepth - 1; ++k) fetch(P.row + k * P.step, o + k * step_o, k);
  int parity = 0, slot = 0;
  for (long long lead = P.lead, row = P.row; lead < a.B;
       lead += P.step, row += P.step, o += step_o, parity ^= 1, slot = slot + 1 == kDepth ? 0 : slot + 1) {
    P.recompute();
    const bool on = row < a.B;
    fetch(row + (kDepth - 1) * P.step, o + (kDepth - 1) * step_o, slot == 0 ? kDepth - 1 : slot - 1);  // the row before's slot
    copy_wait<kDepth - 1>();
    const uint4 *r_dy = ring + slot * streams * words, *r_h = r_dy + words, *r_dh = r_h + words;
    F<V> s = fill<V>(0.0f), d = s;
#pragma unroll
    for (int i = 0; i < NWD; ++i) {
      const F<V> vh = P.own(unpack<T, V>(r_h[i * g.NT]), i), vg = P.own(unpack<T, V>(r_dy[i * g.NT]), i);
      s = fma(vh, vh, s);
      d = fma(mul(vg, unpack<T, V>(wt[i])), vh, d);
    }
    float z[2] = {across(s), across(d)};
    P.reduce(z, buf[parity], [](float p, float q) { return p + q; });
    const float r1 = inverse_rms(z[0], a.inv_C, a.eps);
    const F<V> r = fill<V>(r1), k = fill<V>(-(z[1] * a.inv_C * r1) * r1 * r1);
    if (NWD > 2) asm volatile("" ::: "memory");  // the second pass reads the ring again: the registers are dweight's
    if (on) {
#pragma unroll
      for (int i = 0; i < NWD; ++i) {
        const F<V> vh = P.own(unpack<T, V>(r_h[i * g.NT]), i), rg = mul(P.own(unpack<T, V>(r_dy[i * g.NT]), i), r);
        F<V> d = mul(vh, k);
        if (dh) d = add(d, unpack<T, V>(r_dh[i * g.NT]));
        d = fma(rg, unpack<T, V>(wt[i]), d);
        P.write(a.dx, o, i, packed<T, V>(d));
        dw[i] = fma(rg, vh, dw[i]);
      }
    }
  }
  if (!a.part) return;
  // this CTA's sums over its rows: the teams of a warp, then unit after unit
  copy_wait<0>();
  float* sum = (float*)smem;
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += g.NT) sum[c] = 0.0f;
#pragma unroll
  for (int i = 0; i < NWD; ++i)
    for (int k = 16; k >= P.LANES; k >>= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) dw[i].v[e] += __shfl_xor_sync(0xffffffffu, dw[i].v[e], k);
  const int unit = P.LANES < 32 ? threadIdx.x / 32 : P.team, units = P.LANES < 32 ? g.NT / 32 : g.NT / P.LANES;
  const bool writes = P.LANES >= 32 || (threadIdx.x & 31) < P.LANES;
  for (int t = 0; t < units; ++t) {
    __syncthreads();
    if (t == unit && writes)
#pragma unroll
      for (int i = 0; i < NWD; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (P.in(i, e)) sum[P.at(i) + e] += dw[i].v[e];
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.C; c += g.NT) a.part[(long long)blockIdx.x * a.C + c] = sum[c];
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

bool plan_rows(int B, int C, int es, bool forward, Rows* g) {
  const int V = 16 / es, words = (C + V - 1) / V + (C % V ? 1 : 0);  // of a row, with a partial one at each end
  g->period = V / gcd(C, V);
  // Words to a thread: 4, in the gradient 2 (16384 rows of 2048 bf16 45.1 us, with 4
  // words 47.6; 8599 rows of 6164 133 and 164); one for short rows, and for few rows,
  // so that a call spreads over the SMs; more where the largest team needs it.  The
  // gradient takes pairs of smaller CTAs where a team fits one.
  const bool few = (long long)B * words <= 2LL * kSMs * kThreads && words <= kThreads;
  g->NWD = few || words <= 8 ? 1 : !forward && words <= 2 * kThreads ? 2 : words <= 4 * kThreads ? 4 : 8;
  const int threads = !forward && words <= g->NWD * kThreads / 2 ? kThreads / 2 : kThreads;
  if (words > g->NWD * kThreads || (!forward && es == 2 && g->NWD == 8)) return false;
  g->LANES = 1;
  while (g->LANES * g->NWD < words) g->LANES *= 2;
  g->U = g->LANES < 32 ? 32 / g->LANES : 1;
  const int unit_threads = g->LANES < 32 ? 32 : g->LANES;
  const long long wanted = ((long long)B + g->U - 1) / g->U;  // units, one row each
  const int per_sm = threads < kThreads || (forward && g->NWD == 1) ? 2 : 1;  // CTAs of `threads` threads, by their registers
  g->NT = threads;
  while (g->NT > unit_threads && g->NT > 128 && wanted * unit_threads < (long long)kSMs * g->NT) g->NT /= 2;
  const int per_cta = g->NT / unit_threads;
  long long units = min((wanted + g->period - 1) / g->period * g->period, (long long)kSMs * per_sm * (threads / g->NT) * per_cta);
  // whole CTAs, and a multiple of period
  const int lcm = per_cta / gcd(per_cta, g->period) * g->period;
  units = (units + lcm - 1) / lcm * lcm;
  g->units = (int)units;
  // CTAs up to the last unit that has a row
  const long long span = (long long)g->period * g->U, turn = (B - 1) / span, rho = B - 1 - turn * span;
  const long long used = turn * g->period + min((long long)g->period - 1, rho) + 1;
  g->grid = (int)((min(units, used) + per_cta - 1) / per_cta);
  return true;
}

template <typename T, int NWD, bool Q, bool WHOLE>
int launch_rows(const NormArgs& a, const Rows& g, int qmode, cudaStream_t st) {
  const size_t smem = (size_t)ahead_of(NWD) * g.NT * NWD * 16 * (a.res ? 2 : 1) +
                      (Q && qmode == kAtomic ? (size_t)(g.NT / g.LANES) * a.NG * 4 : 0);
  if (smem > kMaxSmem - kStaticSmem) return DISCO_ERR_UNSUPPORTED;
  return launch_grid(norm_rows_kernel<T, NWD, Q, WHOLE>, g.grid, g.NT, smem, st, "norm_rows_kernel", a, g, qmode);
}

template <typename T, bool Q>
int norm_rows(const NormArgs& a, cudaStream_t st) {
  Rows g;
  constexpr int V = 16 / (int)sizeof(T);
  if (!plan_rows(a.B, a.C, (int)sizeof(T), true, &g)) return DISCO_ERR_UNSUPPORTED;
  int qmode = kRow;
  if (Q && a.NG > 1) {
    const int gw = a.G / V;
    qmode = a.C % V == 0 && a.G % V == 0 && (gw & (gw - 1)) == 0 && gw <= min(g.LANES, 32) ? kLanes : kAtomic;
  }
  const bool whole = a.C % V == 0 && qmode != kAtomic;
  if (g.NWD == 1)
    return whole ? launch_rows<T, 1, Q, true>(a, g, qmode, st) : launch_rows<T, 1, Q, false>(a, g, qmode, st);
  if (g.NWD == 4)
    return whole ? launch_rows<T, 4, Q, true>(a, g, qmode, st) : launch_rows<T, 4, Q, false>(a, g, qmode, st);
  return launch_rows<T, 8, Q, false>(a, g, qmode, st);
}

template <typename T, int NWD, bool WHOLE>
int launch_bwd_rows(const NormBwdArgs& a, const Rows& g, cudaStream_t st) {
  const size_t ring = (size_t)depth_of(NWD) * g.NT * NWD * 16 * (a.dh ? 3 : 2), sums = a.part ? (size_t)a.C * 4 : 0;
  return launch_grid(norm_bwd_rows_kernel<T, NWD, WHOLE>, g.grid, g.NT, ring > sums ? ring : sums, st,
                     "norm_bwd_rows_kernel", a, g);
}

template <typename T>
int norm_bwd_rows(const NormBwdArgs& a, cudaStream_t st) {
  Rows g;
  if (!plan_rows(a.B, a.C, (int)sizeof(T), false, &g)) return DISCO_ERR_UNSUPPORTED;
  if constexpr (sizeof(T) == 4)
    if (g.NWD == 8) return launch_bwd_rows<T, 8, false>(a, g, st);
  const bool whole = g.period == 1;
  if (g.NWD == 1) return whole ? launch_bwd_rows<T, 1, true>(a, g, st) : launch_bwd_rows<T, 1, false>(a, g, st);
  if (g.NWD == 2) return whole ? launch_bwd_rows<T, 2, true>(a, g, st) : launch_bwd_rows<T, 2, false>(a, g, st);
  return whole ? launch_bwd_rows<T, 4, true>(a, g, st) : launch_bwd_rows<T, 4, false>(a, g, st);
}

}  // namespace

int norm_by_rows(const NormArgs& a, disco_dtype dtype, cudaStream_t st) {
  int rc = DISCO_OK;
#define CALL(T) rc = a.q ? norm_rows<T, true>(a, st) : norm_rows<T, false>(a, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

int norm_bwd_by_rows(const NormBwdArgs& a, disco_dtype dtype, cudaStream_t st) {
  int rc = DISCO_OK;
#define CALL(T) rc = norm_bwd_rows<T>(a, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

int norm_bwd_rows_parts(int B, int C, int es) {
  Rows g;
  return plan_rows(B, C, es, false, &g) ? g.grid : 0;
}

}  // namespace norm
}  // namespace disco
