// disco_i8_tc.cuh -- the integer products and their gradients on the tensor cores
// (disco_i8_mm.cuh describes them).
//
//   out[z][m][n] = rs[m] cs[n] sum_{r, k} A(m, k) B(n, k)
//
// sm_103a's tensor cores have no 8-bit integer form worth the name, so integers
// become fp16 (or the tensors' 16-bit type, where a scale belongs to k) on the way into shared
// memory: fp16 holds -128 .. 127, their products are exact, and sums are fp32.
// Persistent kernel of tiles of 128 m x NB n (NB <= 256), 64 k to a stage, four stages:
//   warps 0-3    epilogue: tcgen05.ld, scales, rounding, stores coalesced along n
//   warps 4-11   loaders: 16 bytes of integers from memory to a thread and unit, one
//                step ahead in registers, to 16 bits, into the swizzled stage
//   warp 12      MMA issuer (one thread); two accumulators of NB TMEM columns, so
//                the epilogue of a tile overlaps the main loop of the next
//   warp 13      TMA of an operand that is 16-bit in memory
// Both operands lie in the stage as lines of 64 elements (128 bytes, 128-byte
// swizzle): element k .. k + 63 of one m or n where k is the contiguous direction
// in memory, else (MN-major) 64 neighbouring m or n of one k.  So no operand is ever transposed.
// Rows off 16-byte alignment (ALN false) are read in aligned 16-byte words and
// shifted in registers; a thread's shift stays the same over a tile.
// All mbarrier waits are bounded (time-out -> status flag, abort).
#pragma once

#include <cudaTypedefs.h>

#include "disco_i8_mm.cuh"
#include "disco_umma.cuh"

namespace disco {
namespace i8 {

constexpr int kEpiWarps = 4, kLoadWarps = 8;  // 14 warps: up to 128 registers a thread
constexpr int kMmaWarp = kEpiWarps + kLoadWarps, kTmaWarp = kMmaWarp + 1;
constexpr int kTcThreads = 32 * (kTmaWarp + 1);
constexpr int kLoaders = 32 * kLoadWarps;
constexpr int kBM = 128, kBK = 64, kStages = 4, kNBMax = 256;
constexpr uint32_t kABytes = kBM * kBK * 2, kStageBytes = kABytes + kNBMax * kBK * 2;
constexpr uint32_t kStagePitch = 80;                       // bytes of a row of the epilogue's staging: 64 and 16 against bank conflicts
constexpr uint32_t kEpiBytes = 32 * kStagePitch;           // of a warp
constexpr size_t kTcSmem = 1024 + (size_t)kStages * kStageBytes + kEpiWarps * (kEpiBytes + 128) + 256;
constexpr uint32_t kWaitLimit = 1u << 24;
constexpr int kStatusI8Timeout = 1 << 6;

static __device__ int g_i8_status = 0;  // one per translation unit
__device__ __forceinline__ void i8_flag() { atomicOr(&g_i8_status, kStatusI8Timeout); }

// How an operand lies in memory and what becomes of it.
//   ES: bytes of an element; KM: k is the contiguous direction
//   SC: 0 no scale; else integers times ks[k], in the tensors' type
template <int ES_, bool KM_, int SC_>
struct Form {
  static constexpr int ES = ES_, SC = SC_;
  static constexpr bool KM = KM_;
  static constexpr int UPL = ES == 1 ? 4 : 8;    // 16-byte units of a line of 64 elements
  static constexpr int LPI = kLoaders / UPL;     // lines that the loaders take at a time
};

__device__ __forceinline__ uint64_t tc_desc(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(lbo >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ uint4 ldg16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// The aligned word at p, zeros from `end` on.
__device__ __forceinline__ uint4 ldg16_to(const uint8_t* p, const uint8_t* end) {
  if (p + 16 <= end) return ldg16(p);
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (p + i < end) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Up to 16 bytes of a line as they come from memory.
template <bool ALN>
struct Unit {
  uint4 lo, hi;
};
template <>
struct Unit<true> {
  uint4 lo;
};

template <bool ALN>
__device__ __forceinline__ void load_unit(Unit<ALN>& u, const uint8_t* p, int nb, const uint8_t* base, const uint8_t* end) {
  u.lo = make_uint4(0, 0, 0, 0);
  if constexpr (ALN) {
    if (nb > 0 && DISCO_IN_BOUNDS(p >= base && p + 16 <= end)) u.lo = ldg16(p);
  } else {
    u.hi = make_uint4(0, 0, 0, 0);
    const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    const uint8_t* c = p - sh;
    if (nb > 0 && DISCO_IN_BOUNDS(c >= base && c < end)) {
      u.lo = ldg16_to(c, end);
      if (sh + nb > 16 && DISCO_IN_BOUNDS(c + 16 < end)) u.hi = ldg16_to(c + 16, end);
    }
  }
}

// Its nb bytes, zeros behind them.
template <bool ALN>
__device__ __forceinline__ uint4 unit_bytes(const Unit<ALN>& u, int sh, int nb) {
  if constexpr (ALN) {
    return u.lo;
  } else {
    uint32_t w[8] = {u.lo.x, u.lo.y, u.lo.z, u.lo.w, u.hi.x, u.hi.y, u.hi.z, u.hi.w};
    if (sh & 8)
#pragma unroll
      for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    if (sh & 4)
#pragma unroll
      for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i] = __funnelshift_r(w[i], w[i + 1], 8 * (sh & 3));
      const int left = nb - 4 * i;  // bytes of this word that belong to the line
      if (left < 4) o[i] = left <= 0 ? 0 : o[i] & (0xffffffffu >> (32 - 8 * left));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// 4 integers to 4 fp16 values: 1024 + (q + 128) by the exponent's bits, less 1152; exact.
__device__ __forceinline__ uint2 to_half4(uint32_t w) {
  w ^= 0x80808080u;
  const __half2 off = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
  __half2 a = __hsub2(*reinterpret_cast<__half2*>(&lo), off), b = __hsub2(*reinterpret_cast<__half2*>(&hi), off);
  return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
}
// 4 integers times scales to 4 values of the type, rounded once.
template <bool HALF>
__device__ __forceinline__ uint2 to_scaled4(uint32_t w, float s0, float s1, float s2, float s3) {
  w ^= 0x80808080u;
  return make_uint2(pack2_16(from_byte(w, 0) * s0, from_byte(w, 1) * s1, HALF),
                    pack2_16(from_byte(w, 2) * s2, from_byte(w, 3) * s3, HALF));
}

// One operand's share of a loader thread.
template <class F, bool ALN, int LINES>
struct Loader {
  static constexpr int NU = LINES / F::LPI;  // units of this thread in a stage, at most
  const uint8_t *base, *end, *row;           // the tensor; this slice's
  long long ld;
  int u, l0;           // unit of a line, first line
  long long i0;        // first m or n of the tile
  int ileft;           // m or n of the tile inside the tensor

  __device__ __forceinline__ void init(const Operand& o, const uint8_t* e, int t) {
    base = (const uint8_t*)o.p, end = e, ld = o.ld * F::ES;
    u = t % F::UPL, l0 = t / F::UPL;
  }
  __device__ __forceinline__ void tile(const Operand& o, long long z, long long r, long long first, long long I) {
    row = base + (z * o.z + r * o.r) * F::ES;
    i0 = first;
    ileft = (int)min(I - first, (long long)LINES);
  }
  // where unit j of the step lies, and how many of its bytes are inside
  __device__ __forceinline__ const uint8_t* at(int j, long long k0, int kleft, int* nb) const {
    const int line = l0 + j * F::LPI;
    if constexpr (F::KM) {
      *nb = line < ileft ? min(16, kleft * F::ES - 16 * u) : 0;
      return row + (i0 + line) * ld + k0 * F::ES + 16 * u;
    } else {
      const int box = line >> 6, kk = line & 63;
      *nb = kk < kleft ? min(16, (ileft - 64 * box) * F::ES - 16 * u) : 0;
      return row + (k0 + kk) * ld + (i0 + 64 * box) * F::ES + 16 * u;
    }
  }
  // units j0 .. j0 + N - 1 of the thread
  template <int N>
  __device__ __forceinline__ void fetch(Unit<ALN> (&w)[N], int j0, long long k0, int kleft, int lines) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if ((j0 + j) * F::LPI < lines) {
        int nb;
        const uint8_t* p = at(j0 + j, k0, kleft, &nb);
        load_unit<ALN>(w[j], p, nb, base, end);
      }
  }
  // all units, four at a time
  template <bool HALF>
  __device__ __forceinline__ void copy(uint8_t* stage, const float* ks, long long k0, int kleft, int lines) const {
    constexpr int N = NU < 4 ? NU : 4;
#pragma unroll 1
    for (int j0 = 0; j0 * F::LPI < lines; j0 += N) {
      Unit<ALN> w[N];
      fetch(w, j0, k0, kleft, lines);
      put<HALF>(w, j0, stage, ks, k0, kleft, lines);
    }
  }
  template <bool HALF, int N>
  __device__ __forceinline__ void put(const Unit<ALN> (&w)[N], int j0, uint8_t* stage, const float* ks, long long k0, int kleft, int lines) const {
    float s[16];
    if constexpr (F::SC && F::KM) {  // all lines share the step's scales
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = 16 * u + i < kleft ? __ldg(ks + k0 + 16 * u + i) : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
      if ((j0 + j) * F::LPI < lines) {
        const int line = l0 + (j0 + j) * F::LPI;
        int nb = 16, sh = 0;
        if constexpr (!ALN) sh = (int)(reinterpret_cast<uintptr_t>(at(j0 + j, k0, kleft, &nb)) & 15);
        const uint4 v = unit_bytes<ALN>(w[j], sh, nb);
        uint8_t* d = stage + line * 128;
        const int x = line & 7;
        if constexpr (F::ES == 2) {
          *reinterpret_cast<uint4*>(d + ((u ^ x) << 4)) = v;
        } else {
          uint2 a, b, c, e;
          if constexpr (F::SC == 0) {
            a = to_half4(v.x), b = to_half4(v.y), c = to_half4(v.z), e = to_half4(v.w);
          } else if constexpr (F::KM) {
            a = to_scaled4<HALF>(v.x, s[0], s[1], s[2], s[3]), b = to_scaled4<HALF>(v.y, s[4], s[5], s[6], s[7]);
            c = to_scaled4<HALF>(v.z, s[8], s[9], s[10], s[11]), e = to_scaled4<HALF>(v.w, s[12], s[13], s[14], s[15]);
          } else {
            const int kk = line & 63;
            const float f = kk < kleft ? __ldg(ks + k0 + kk) : 0.0f;
            a = to_scaled4<HALF>(v.x, f, f, f, f), b = to_scaled4<HALF>(v.y, f, f, f, f);
            c = to_scaled4<HALF>(v.z, f, f, f, f), e = to_scaled4<HALF>(v.w, f, f, f, f);
          }
          *reinterpret_cast<uint4*>(d + (((2 * u) ^ x) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
          *reinterpret_cast<uint4*>(d + (((2 * u + 1) ^ x) << 4)) = make_uint4(c.x, c.y, e.x, e.y);
        }
      }
  }
};

__device__ __forceinline__ void tc_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tc_tma_3d(void* dst, const CUtensorMap* map, int c0, int c1, int c2, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// FA, FB: the operands' forms; HALF: 16-bit operands are fp16; ALN: every row of
// every operand starts on 16 bytes.  `map`: the 16-bit operand's (ALN only).
template <class FA, class FB, bool HALF, bool ALN>
__global__ void __launch_bounds__(kTcThreads, 1) i8_tc_kernel(const __grid_constant__ CUtensorMap map, const TcArgs a) {
  constexpr bool kTma = ALN && (FA::ES == 2 || FB::ES == 2);
  constexpr bool kLoadA = !(kTma && FA::ES == 2), kLoadB = !(kTma && FB::ES == 2);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = smem + kStages * kStageBytes;
  float* colscale = reinterpret_cast<float*>(staging + kEpiWarps * kEpiBytes);  // [kEpiWarps][32]
  uint64_t* full = reinterpret_cast<uint64_t*>(colscale + kEpiWarps * 32);
  uint64_t *empty = full + kStages, *accf = empty + kStages, *acce = accf + 2;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(acce + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kLoadWarps + (kTma ? 1 : 0));
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], kEpiWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tslot, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;

  // tile t: m fastest (CTAs side by side share the n tile in L2), then n, z and the split
  struct Tile {
    long long m0, n0, z, q0, q1;
    int sp;
  };
  auto tile_of = [&](long long t) {
    Tile c;
    c.m0 = t % a.mt * kBM;
    t /= a.mt;
    c.n0 = t % a.nt * a.NB;
    t /= a.nt;
    c.z = t % a.m.Z;
    c.sp = (int)(t / a.m.Z);
    c.q0 = a.steps * c.sp / a.nsplit;
    c.q1 = a.steps * (c.sp + 1) / a.nsplit;
    return c;
  };

  if (warp >= kEpiWarps && warp < kMmaWarp) {
    // ------------------------------------------------------------ loaders --
    Loader<FA, ALN, kBM> la;
    Loader<FB, ALN, kNBMax> lb;
    la.init(a.m.A, a.enda, tid - 32 * kEpiWarps);
    lb.init(a.m.B, a.endb, tid - 32 * kEpiWarps);
    // rows off alignment are not held a step ahead: two words to a unit would not fit the registers
    constexpr bool kAheadA = kLoadA && ALN, kAheadB = kLoadB && ALN;
    using UA = Unit<ALN>[Loader<FA, ALN, kBM>::NU];
    using UB = Unit<ALN>[Loader<FB, ALN, kNBMax>::NU];
    struct Pos {
      long long t, q, k0;
      long long q1;
      const float *ksa, *ksb;  // the slice's scales on k
      int kleft;
    };
    auto place = [&](Pos& p, bool fresh) {  // loaders at step p.q of tile p.t
      const long long r = a.m.R == 1 ? 0 : p.q / a.nkp, kc = p.q - r * a.nkp;
      p.k0 = kc * kBK;
      p.kleft = (int)min(a.m.K - p.k0, (long long)kBK);
      if (fresh || kc == 0) {
        const Tile c = tile_of(p.t);
        la.tile(a.m.A, c.z, r, c.m0, a.m.M);
        lb.tile(a.m.B, c.z, r, c.n0, a.m.N);
        p.ksa = FA::SC ? a.m.A.ks + r * a.m.A.ks_r : nullptr;
        p.ksb = FB::SC ? a.m.B.ks + r * a.m.B.ks_r : nullptr;
      }
    };
    auto start = [&](Pos& p, long long t) {
      p.t = t;
      if (t >= a.tiles) return;
      const Tile c = tile_of(t);
      p.q = c.q0, p.q1 = c.q1;
      place(p, true);
    };
    auto advance = [&](Pos& p) {
      if (++p.q == p.q1) start(p, p.t + gridDim.x);
      else place(p, false);
    };
    int i = 0;
    bool ok = true;
    auto store = [&](const Pos& p, const UA& ua, const UB& ub) {  // step p, whose units were fetched before
      const int s = i % kStages;
      if (i >= kStages) ok = mbar_wait(&empty[s], ((i / kStages) - 1) & 1, kWaitLimit);
      ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
      if (!ok) return;
      uint8_t* sa = smem + s * kStageBytes;
      if constexpr (kAheadA) la.template put<HALF>(ua, 0, sa, p.ksa, p.k0, p.kleft, kBM);
      if constexpr (kAheadB) lb.template put<HALF>(ub, 0, sa + kABytes, p.ksb, p.k0, p.kleft, a.NB);
      if constexpr (kLoadA && !kAheadA) la.template copy<HALF>(sa, p.ksa, p.k0, p.kleft, kBM);
      if constexpr (kLoadB && !kAheadB) lb.template copy<HALF>(sa + kABytes, p.ksb, p.k0, p.kleft, a.NB);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[s]);
      ++i;
    };
    auto fetch = [&](const Pos& p, UA& ua, UB& ub) {
      if constexpr (kAheadA) la.fetch(ua, 0, p.k0, p.kleft, kBM);
      if constexpr (kAheadB) lb.fetch(ub, 0, p.k0, p.kleft, a.NB);
    };
    Pos cur, nxt;
    UA ua0, ua1;
    UB ub0, ub1;
    start(cur, blockIdx.x);
    if constexpr (ALN) {
      if (cur.t < a.tiles) fetch(cur, ua0, ub0);
      while (ok && cur.t < a.tiles) {
        nxt = cur;
        advance(nxt);
        if (nxt.t < a.tiles) fetch(nxt, ua1, ub1);
        store(cur, ua0, ub0);
        if (!ok || nxt.t >= a.tiles) break;
        cur = nxt;
        advance(cur);
        if (cur.t < a.tiles) fetch(cur, ua0, ub0);
        store(nxt, ua1, ub1);
      }
    } else {
      for (; ok && cur.t < a.tiles; advance(cur)) store(cur, ua0, ub0);
    }
    if (!ok) {
      i8_flag();
      *abort_flag = 1;
    }
  } else if (warp == kTmaWarp) {
    // ---------------------------------------------- TMA of a 16-bit operand --
    if constexpr (kTma) {
      if (lane == 0) {
        constexpr bool kIsA = FA::ES == 2;
        constexpr bool kKM = kIsA ? FA::KM : FB::KM;
        const int lines = kIsA ? kBM : a.NB;
        int i = 0;
        bool ok = true;
        for (long long t = blockIdx.x; t < a.tiles && ok; t += gridDim.x) {
          const Tile c = tile_of(t);
          const long long i0 = kIsA ? c.m0 : c.n0, I = kIsA ? a.m.M : a.m.N;
          for (long long q = c.q0; q < c.q1; ++q, ++i) {
            const int s = i % kStages;
            if ((i >= kStages && !mbar_wait(&empty[s], ((i / kStages) - 1) & 1, kWaitLimit)) || *abort_flag) {
              ok = false;
              break;
            }
            const long long r = q / a.nkp, k0 = (q - r * a.nkp) * kBK, zr = a.m.R == 1 ? c.z : r;
            uint8_t* d = smem + s * kStageBytes + (kIsA ? 0 : kABytes);
            tc_expect_tx(&full[s], (uint32_t)lines * 128);
            // boxes start inside the operand; past its ends the copy engine writes zeros
            if (!DISCO_IN_BOUNDS(i0 >= 0 && i0 < I && k0 >= 0 && k0 < a.m.K && zr >= 0 && zr < (long long)a.m.Z * a.m.R)) {
              mbar_complete_tx(&full[s], (uint32_t)lines * 128);
              continue;
            }
            if (kKM) {
              tc_tma_3d(d, &map, (int)k0, (int)i0, (int)zr, &full[s]);
            } else {
              for (int b = 0; b < lines / 64; ++b) tc_tma_3d(d + b * 8192, &map, (int)i0 + 64 * b, (int)k0, (int)zr, &full[s]);
            }
          }
        }
        if (!ok) {
          i8_flag();
          *abort_flag = 1;
        }
        // the copies in flight end before the CTA does
        for (int back = 1; back <= kStages && i - back >= 0 && !ok; ++back)
          mbar_wait(&full[(i - back) % kStages], ((i - back) / kStages) & 1, 1u << 16);
      }
    }
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------- MMA issuer --
    if (lane == 0) {
      // without scales on k both operands are fp16 whatever the output
      constexpr bool kHalfOp = HALF || (FA::ES == 1 && FB::ES == 1);
      const uint32_t idesc = idesc_16_f32(kBM, a.NB, kHalfOp) | (FA::KM ? 0u : 1u << 15) | (FB::KM ? 0u : 1u << 16);
      int i = 0, tl = 0;
      bool ok = true;
      for (long long t = blockIdx.x; t < a.tiles && ok; t += gridDim.x, ++tl) {
        const Tile c = tile_of(t);
        const int ab = tl & 1;
        if (tl >= 2 && !mbar_wait(&acce[ab], ((tl >> 1) - 1) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (long long q = c.q0; q < c.q1; ++q, ++i) {
          const int s = i % kStages;
          if (!mbar_wait(&full[s], (i / kStages) & 1, kWaitLimit) || *abort_flag) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * kStageBytes), sb = sa + kABytes;
#pragma unroll
          for (int ks = 0; ks < kBK / 16; ++ks) {
            // 16 k: 32 bytes of every line (k contiguous), or 16 lines; boxes of 64 m or n are 8 KB apart
            const uint64_t ad = FA::KM ? tc_desc(sa + ks * 32, 16) : tc_desc(sa + ks * 2048, 8192);
            const uint64_t bd = FB::KM ? tc_desc(sb + ks * 32, 16) : tc_desc(sb + ks * 2048, 8192);
            umma_bf16(tmem + ab * kNBMax, ad, bd, idesc, (q > c.q0 || ks > 0) ? 1u : 0u);
          }
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&accf[ab]);
      }
      if (!ok) {
        i8_flag();
        *abort_flag = 1;
        if (i > 0) mbar_wait(&empty[(i - 1) % kStages], ((i - 1) / kStages) & 1, kWaitLimit);
      }
    }
  } else if (warp < kEpiWarps) {
    // ----------------------------------------------------------- epilogue --
    const int q4 = warp;  // TMEM lanes 32 q4 ..
    uint8_t* stg = staging + warp * kEpiBytes;
    const bool split = a.part != nullptr;
    const int type = split ? DISCO_F32 : a.out_type, eb = type == DISCO_F32 ? 4 : 2;
    int tl = 0;
    for (long long t = blockIdx.x; t < a.tiles; t += gridDim.x, ++tl) {
      const Tile c = tile_of(t);
      const int ab = tl & 1;
      float* cs = colscale + warp * 32;
      const bool scaled = !split && a.m.cs;
      // scale of column c0 + lane, fetched a chunk ahead
      auto column = [&](int col) { return scaled && c.n0 + col < a.m.N ? __ldg(a.m.cs + c.z * a.m.cs_z + c.n0 + col) : 0.0f; };
      float next = column(lane);
      const long long row0 = c.m0 + q4 * 32;
      const float rs = !split && a.m.rs && row0 + lane < a.m.M ? a.m.rs[row0 + lane] : 1.0f;
      bool fin = mbar_wait(&accf[ab], (tl >> 1) & 1, kWaitLimit);
      fin = __all_sync(0xffffffffu, fin) && !*abort_flag;
      if (!fin) {
        if (lane == 0) i8_flag();
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const int rows = (int)min(a.m.M - row0, 32LL);  // of this warp, may be negative
      uint8_t* out = (uint8_t*)(split ? (void*)a.part : a.m.out) +
                     (((c.sp * (long long)a.m.Z + c.z) * a.m.M + row0) * a.m.N + c.n0) * eb;
      const long long pitch = a.m.N * eb;
      const int cols = (int)min(a.m.N - c.n0, (long long)a.NB);
      for (int c0 = 0; c0 < cols; c0 += 32) {
        uint32_t v[32];
        tmem_ld32(tmem + ab * kNBMax + ((uint32_t)(q4 * 32) << 16) + c0, v);
        if (scaled) {
          cs[lane] = next;
          __syncwarp();
          next = column(c0 + 32 + lane);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(cs + e);
            v[e] = __float_as_uint(__uint_as_float(v[e]) * f.x * rs);
            v[e + 1] = __float_as_uint(__uint_as_float(v[e + 1]) * f.y * rs);
            v[e + 2] = __float_as_uint(__uint_as_float(v[e + 2]) * f.z * rs);
            v[e + 3] = __float_as_uint(__uint_as_float(v[e + 3]) * f.w * rs);
          }
        }
        // 64 bytes of each of the warp's 32 rows at a time through shared memory
        auto emit = [&](int w0, int n) {  // n columns from c0 + w0 are staged
          __syncwarp();
          const int left = min(n, cols - c0 - w0);
          uint8_t* o = out + (long long)(c0 + w0) * eb;
          if (a.vec) {
#pragma unroll
            for (int h = 0; h < 4; ++h) {
              const int idx = lane + 32 * h, row = idx >> 2, seg = idx & 3;
              if (row < rows && seg * 16 < left * eb)
                *reinterpret_cast<uint4*>(o + row * pitch + seg * 16) = *reinterpret_cast<const uint4*>(stg + row * kStagePitch + seg * 16);
            }
          } else if (eb == 2) {
            if (lane < left)
#pragma unroll 4
              for (int row = 0; row < rows; ++row)
                *reinterpret_cast<uint16_t*>(o + row * pitch + lane * 2) = *reinterpret_cast<const uint16_t*>(stg + row * kStagePitch + lane * 2);
          } else {
            if ((lane & 15) < left)
#pragma unroll 4
              for (int row = lane >> 4; row < rows; row += 2)
                *reinterpret_cast<uint32_t*>(o + row * pitch + (lane & 15) * 4) =
                    *reinterpret_cast<const uint32_t*>(stg + row * kStagePitch + (lane & 15) * 4);
          }
          __syncwarp();
        };
        uint4* d = reinterpret_cast<uint4*>(stg + lane * kStagePitch);
        if (type == DISCO_F32) {
#pragma unroll
          for (int g = 0; g < 4; ++g) d[g] = make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
          emit(0, 16);
          if (c0 + 16 < cols) {
#pragma unroll
            for (int g = 0; g < 4; ++g) d[g] = make_uint4(v[16 + 4 * g], v[17 + 4 * g], v[18 + 4 * g], v[19 + 4 * g]);
            emit(16, 16);
          }
        } else {
          const bool h16 = type == DISCO_F16;
          auto two = [&](int e) { return pack2_16(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), h16); };
#pragma unroll
          for (int g = 0; g < 4; ++g) d[g] = make_uint4(two(8 * g), two(8 * g + 2), two(8 * g + 4), two(8 * g + 6));
          emit(0, 32);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[ab]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- host --------------------------------------------------------------------

inline int tc_encode(CUtensorMap* map, const Operand& o, long long I, long long K, int ZR, int lines, bool f16) {
  static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  if (!enc) return fail(DISCO_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const long long slice = max(o.z, o.r);
  const cuuint64_t dims[3] = {(cuuint64_t)(o.k_major ? K : I), (cuuint64_t)(o.k_major ? I : K), (cuuint64_t)ZR};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * 2, (cuuint64_t)(slice ? slice : o.ld * dims[1]) * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)(o.k_major ? lines : 64), 1}, estr[3] = {1, 1, 1};
  const CUresult cr = enc(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(o.p),
                          dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(DISCO_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)cr);
  return DISCO_OK;
}

template <class FA, class FB, bool HALF, bool ALN>
int tc_launch(const TcArgs& a, cudaStream_t st) {
  CUtensorMap map = {};
  if constexpr (ALN && (FA::ES == 2 || FB::ES == 2)) {
    int rc;
    if (FA::ES == 2) rc = tc_encode(&map, a.m.A, a.m.M, a.m.K, a.m.Z * a.m.R, kBM, HALF);
    else rc = tc_encode(&map, a.m.B, a.m.N, a.m.K, a.m.Z * a.m.R, a.NB, HALF);
    if (rc) return rc;
  }
  auto kern = i8_tc_kernel<FA, FB, HALF, ALN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kTcSmem) != cudaSuccess)
    return check_launch("i8_tc_kernel attribute");
  kern<<<(int)min(a.tiles, (long long)kSMs), kTcThreads, kTcSmem, st>>>(map, a);
  return check_launch("i8_tc_kernel");
}

// This unit's status word (ORed into *v, and optionally cleared).
#define DISCO_I8_STATUS_READER(name)                                                   \
  cudaError_t name(int32_t* v, bool clear) {                                           \
    int32_t t = 0;                                                                     \
    cudaError_t e = cudaMemcpyFromSymbol(&t, i8::g_i8_status, sizeof(int32_t));        \
    if (e == cudaSuccess && clear) {                                                   \
      const int32_t zero = 0;                                                          \
      e = cudaMemcpyToSymbol(i8::g_i8_status, &zero, sizeof(int32_t));                 \
    }                                                                                  \
    *v |= t;                                                                           \
    return e;                                                                          \
  }

}  // namespace i8
}  // namespace disco
