// disco_i8_tc.cuh -- the integer products and their gradients on the tensor cores
// (disco_i8_mm.cuh describes them).
//
//   out[z][m][n] = rs[m] cs[n] sum_{r, k} A(m, k) B(n, k)
//
// sm_103a's tensor cores have no 8-bit integer form worth the name, so integers
// become fp16: it holds -128 .. 127, their products are exact, and sums are fp32.  Where a scale belongs
// to k (both gradients) the integer times its scale is rounded to the tensors' 16-bit type, as a 16-bit operand
// would be (errors sqrt(2) of the output's rounding; a high and a low part would double the matrix work).  A is the activation (8-bit integers,
// converted on the way into shared memory, or 16-bit); B is 16-bit: a weight converted
// once a call into the workspace, or dy.  A tile is 128 m x NB n (NB <= 256), 64 k to a
// stage, so a step converts 128 lines and multiplies 128 by 256: with both operands
// converted in the main loop the product of 16384 rows of 2048 by 2048 took 261 us.
// Measured (GB300, bf16): that product 106 us, 1.30 PFLOP/s, dx 91, dW 132; 512 -> 512
// channels on 360x720 128 us, dx 124, dW 126; 2 x 128 -> 256 on 361x720 85, 68 and 74.
// What the counters say of the large ones, while their CTAs run: 512 channels, the threads' accesses to shared
// memory (converters and epilogue) 80 % of their pipe, the matrix unit 46 %; that product of rows, no unit above
// 60 % (matrix unit 59, accesses 53); its dx, the matrix unit 73 %, 18 TB/s from L2; its dW, 128 tiles on as many of
// the 152 SMs, there the matrix unit 52 %, issue slots 48 %.  Shared memory's banks are read and written a quarter of the
// time each.  Grids of few channels are bound by what a tile costs at least (1.3 us of an SM), those between by HBM.
// Dropped: pairs of CTAs (256 x 256 tiles, half of B each; rows 134 us and dx 118, before the issuing threads were
// elected), and prefetches to L2 four steps ahead (rows 119, dx 184, dW 246).
// Persistent kernel:
//   epilogue     (8 warps; 4 for the weight's gradient, whose tiles are few): tcgen05.ld,
//                scales, rounding, stores along the output's rows
//   converters   (8 warps, idle where both operands are 16-bit): integers from the raw ring, to 16 bits, into the
//                stage.  Two groups take alternate steps, so that one's loads, conversion and
//                fence overlap the other's.  The raw ring has an even number of slots, each always
//                the same group's, and stages are released in order: no waiter is ever two
//                phases ahead of a barrier, where a wait by parity would pass at once.  They
//                convert after the wait for the stage: before it, dW of 512 by 512 channels on 360x720 took 138 us (124)
//   one warp     MMA issuer (one thread); two accumulators of 256 TMEM columns, so
//                the epilogue of a tile overlaps the main loop of the next.  Of narrow tiles
//                four or eight, and each half of eight epilogue warps takes every second tile
//   two warps    TMA of B and of A: into the stage (16-bit) or the raw ring (integers)
// Both operands lie in the stage as lines of 64 elements (128 bytes, 128-byte
// swizzle): element k .. k + 63 of one m or n where k is the contiguous direction
// in memory, else (MN-major) 64 neighbouring m or n of one k.  So no operand is ever transposed.
// Operands whose rows do not start on 16 bytes are laid out anew in the workspace first
// (disco_i8_mm.cu): with the converters reading and shifting their words instead, dx of
// 512 -> 512 on 259199 pixels took 326 us and dW 676; copy and product take 242 and 284.
// All mbarrier waits are bounded (time-out -> status flag, abort).
#pragma once

#include <cudaTypedefs.h>

#include "disco_i8_mm.cuh"
#include "disco_umma.cuh"

namespace disco {
namespace i8 {

constexpr int kBM = 128, kBK = 64, kNBMax = 256;
constexpr uint32_t kABytes = kBM * kBK * 2, kBBytes = kNBMax * kBK * 2;
constexpr uint32_t kWaitLimit = 1u << 24;  // the longest wait spans the kPartSteps of a tile's part, below a millisecond
constexpr int kStatusI8Timeout = 1 << 6;

static __device__ int g_i8_status = 0;  // one per translation unit
__device__ __forceinline__ void i8_flag() { atomicOr(&g_i8_status, kStatusI8Timeout); }

// How A lies in memory and what becomes of it.
//   ES: bytes of an element; KM: k is the contiguous direction
//   SC: 0 no scale; else integers times ks[k], in the tensors' type
template <int ES_, bool KM_, int SC_>
struct Form {
  static constexpr int ES = ES_, SC = SC_;
  static constexpr bool KM = KM_;
};


// What the forms make of warps and shared memory (227 KB).
template <class FA>
struct Plan {
  static constexpr bool kRaw = FA::ES == 1;  // A by TMA into the raw ring
  static constexpr int kEpi = FA::SC ? 4 : 8, kConv = kRaw ? 8 : 4;
  static constexpr int kMmaWarp = kEpi + kConv, kThreads = 32 * (kMmaWarp + 3);
  static constexpr int kGroups = 2, kGroupWarps = kConv / kGroups;
  // Slots of B (and barriers of a step), of A, and of the raw ring.  A slot of A waits for the
  // products of step i - kAs by that step's barrier; its waiter has seen step i - 2 - kAs
  // end, so the barrier is never a phase behind.  B comes from memory or L2 and wants the
  // lead: with 3, 3 and 6 slots dW of 16384 rows of 2048 by 2048 took 171 us (144 then), 512 -> 512 on 360x720
  // 136 (128); with 4 of A and 2 raw dW 156.
  static constexpr int kStages = 4, kAs = !kRaw ? 4 : FA::SC ? 3 : 2, kRaws = kRaw ? 4 : 0;
  static constexpr uint32_t kSlot = kBM * kBK;
  // of an epilogue warp: 64 bytes of 32 rows on their way out, the scales of a tile's columns
  static constexpr uint32_t kStaging = 32 * 64, kCols = kRaw && !FA::SC ? kNBMax * 4 : 0;
  static constexpr size_t kSmem = 1024 + (size_t)kAs * kABytes + (size_t)kStages * kBBytes + kRaws * kSlot + kEpi * (kStaging + kCols) + 512;
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  static_assert(kRaws % kGroups == 0, "a slot is always the same group's");
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

// A's share of a converter thread: four 16-byte units of a step.  The raw slot holds 128 lines of
// 64 k, or (MN-major) 64 k of 128 m: whole sectors to a copy's row.  There eight lanes take both
// halves of neighbouring k, which the stage keeps 8 KB apart, so that neither side's
// accesses meet in a bank.
template <class F, int NT>
struct Units {
  static_assert(NT == 128, "the units below");
  static constexpr int N = 4;
  int t, u, l0, h;  // unit of a line; first line (k contiguous) or k

  __device__ __forceinline__ explicit Units(int t) : t(t), u(t % 4), l0(F::KM ? t / 4 : t / 8 * 2 + (t / 4 & 1)), h(t / 4 & 1) {}
  __device__ __forceinline__ int line(int j) const { return F::KM ? l0 + 32 * j : l0 + 32 * (j >> 1) + 64 * (h ^ (j & 1)); }
  __device__ __forceinline__ int raw(int j) const { return F::KM ? t + NT * j : (l0 + 32 * (j >> 1)) * 8 + 4 * (h ^ (j & 1)) + u; }
  // The scales of this thread's units of a step: of 16 k (k contiguous), or of its two k.
  // ks: of the step's first k; the row of scales goes on in zeros to a multiple of 16.
  static constexpr int NS = F::SC == 0 ? 1 : F::KM ? 16 : 2;
  __device__ __forceinline__ void scales(float (&s)[NS], const float* ks, int kleft) const {
    if constexpr (F::SC && F::KM) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 f = 16 * u < kleft ? __ldg(reinterpret_cast<const float4*>(ks + 16 * u + i)) : make_float4(0, 0, 0, 0);
        s[i] = f.x, s[i + 1] = f.y, s[i + 2] = f.z, s[i + 3] = f.w;
      }
    } else if constexpr (F::SC) {
#pragma unroll
      for (int i = 0; i < NS; ++i) s[i] = l0 + 32 * i < kleft ? __ldg(ks + l0 + 32 * i) : 0.0f;
    }
  }
  // unit j into the stage
  template <bool HALF>
  __device__ __forceinline__ void put(const uint4& v, int j, const float (&s)[NS], uint8_t* stage) const {
    const int x = line(j) & 7;
    uint8_t* d = stage + line(j) * 128;
    uint2 a, b, c, e;
    if constexpr (F::SC == 0) {
      a = to_half4(v.x), b = to_half4(v.y), c = to_half4(v.z), e = to_half4(v.w);
    } else if constexpr (F::KM) {
      a = to_scaled4<HALF>(v.x, s[0], s[1], s[2], s[3]), b = to_scaled4<HALF>(v.y, s[4], s[5], s[6], s[7]);
      c = to_scaled4<HALF>(v.z, s[8], s[9], s[10], s[11]), e = to_scaled4<HALF>(v.w, s[12], s[13], s[14], s[15]);
    } else {
      const float f = s[j >> 1];
      a = to_scaled4<HALF>(v.x, f, f, f, f), b = to_scaled4<HALF>(v.y, f, f, f, f);
      c = to_scaled4<HALF>(v.z, f, f, f, f), e = to_scaled4<HALF>(v.w, f, f, f, f);
    }
    *reinterpret_cast<uint4*>(d + (((2 * u) ^ x) << 4)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4*>(d + (((2 * u + 1) ^ x) << 4)) = make_uint4(c.x, c.y, e.x, e.y);
  }
};

// A CTA's tiles: tile t has n fastest (CTAs side by side share A's tile in L2), then m, z
// and the part; the next one is gridDim.x on, by additions (divisions for each tile took a
// third of one of four steps).
struct Walk {
  uint32_t t;
  int n, m, z, sp, dn, dm, dz, dsp;
  __device__ __forceinline__ explicit Walk(const TcArgs& a) {
    t = blockIdx.x;
    split(a, t, &n, &m, &z, &sp);
    split(a, gridDim.x, &dn, &dm, &dz, &dsp);
  }
  __device__ static __forceinline__ void split(const TcArgs& a, uint32_t t, int* n, int* m, int* z, int* sp) {
    uint32_t u = t / a.nt;
    *n = (int)(t - u * a.nt);
    t = u / a.mt;
    *m = (int)(u - t * a.mt);
    u = t / (uint32_t)a.m.Z;
    *z = (int)(t - u * a.m.Z);
    *sp = (int)u;
  }
  __device__ __forceinline__ void next(const TcArgs& a) {
    t += gridDim.x;
    n += dn, m += dm, z += dz, sp += dsp;
    if (n >= (int)a.nt) n -= a.nt, ++m;
    if (m >= (int)a.mt) m -= a.mt, ++z;
    if (z >= a.m.Z) z -= a.m.Z, ++sp;
  }
  __device__ __forceinline__ bool in(const TcArgs& a) const { return t < a.tiles; }
  __device__ __forceinline__ long long m0() const { return (long long)m * kBM; }
  __device__ __forceinline__ long long n0(const TcArgs& a) const { return (long long)n * a.NB; }
};

// Where a converter is: step q of tile t, slice r, chunk kc.
struct Pos {
  Walk w;
  long long q, q1, r, kc;
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

// One thread of a whole warp, for the loops of copies and matrix instructions: the compiler
// knows that it is one.  With lane 0 instead, and ring sizes taken at run time, their threads were
// busy 1000 cycles a step: dx of 16384 rows of 2048 by 2048 took 109 us (91), dW 143 (132).
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// One row on; opaque to the compiler, which would keep 32 rows' addresses in registers.
__device__ __forceinline__ void next_row(uint8_t*& o, long long pitch) { asm volatile("add.s64 %0, %0, %1;" : "+l"(o) : "l"(pitch)); }

// FA: A's form; BKM: B is K-major; HALF: 16-bit operands are fp16; TR: out[z][n][m]
// instead of [m][n].
template <class FA, bool BKM, bool HALF, bool TR>
__global__ void __launch_bounds__(Plan<FA>::kThreads, 1)
    i8_tc_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, const TcArgs a) {
  using C = Plan<FA>;
  constexpr int kMmaWarp = C::kMmaWarp, kTmaBWarp = kMmaWarp + 1, kTmaAWarp = kMmaWarp + 2, kStages = C::kStages, kAs = C::kAs, kRaws = C::kRaws;
  constexpr int kEpiWarps = C::kEpi, kGroups = C::kGroups, kGroupWarps = C::kGroupWarps, kConverters = 32 * kGroupWarps;
  constexpr bool kRaw = C::kRaw, kFit = HALF && (FA::SC || !kRaw);  // kFit: fp16 gradients
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t *bring = smem + kAs * kABytes, *raws = bring + kStages * kBBytes;
  uint8_t* staging = raws + kRaws * C::kSlot;
  uint8_t* colscale = staging + kEpiWarps * C::kStaging;
  uint64_t* full = reinterpret_cast<uint64_t*>(colscale + kEpiWarps * C::kCols);
  uint64_t *empty = full + 4, *accf = empty + 4, *acce = accf + 8, *rawf = acce + 8, *rawe = rawf + 8;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(rawe + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  uint32_t* most = tslot + 2;  // of the scales (Range)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int accs = a.NB <= 64 ? 8 : a.NB <= 128 ? 4 : 2, acc_cols = 512 / accs;  // accumulators, their columns
  const bool turns = kEpiWarps == 8 && accs > 2;                                 // the epilogue's halves take turns
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], (kRaw ? kGroupWarps : 1) + 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 8; ++b) {
      mbar_init(&accf[b], 1);
      mbar_init(&acce[b], turns ? 4 : kEpiWarps);
    }
    for (int r = 0; r < 8; ++r) {
      mbar_init(&rawf[r], 1);
      mbar_init(&rawe[r], kGroupWarps);
    }
    *abort_flag = 0;
    *most = 0;
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
  norm::wait_for_previous();  // the operand that was converted into the workspace
  if constexpr (kFit) {
    const uint32_t m = largest(a.m.range.v, a.m.range.n, tid, C::kThreads);
    if (lane == 0) atomicMax(most, m);
    __syncthreads();
  }

  // reduction steps of a tile's part
  auto first_step = [&](int sp) { return a.nsplit > 1 ? a.steps * sp / a.nsplit : 0; };
  auto last_step = [&](int sp) { return a.nsplit > 1 ? a.steps * (sp + 1) / a.nsplit : a.steps; };

  if (warp >= kEpiWarps && warp < kMmaWarp) {
    // --------------------------------------------------------- converters --
    if constexpr (kRaw) {
      const int group = (warp - kEpiWarps) / kGroupWarps, t0 = tid - 32 * kEpiWarps - group * kConverters;
      using U = Units<FA, kConverters>;
      const U units(t0);
      [[maybe_unused]] const float down = kFit ? fit_down(*most) : 1.0f;
      auto start = [&](Pos& p) {
        p.q = first_step(p.w.sp), p.q1 = last_step(p.w.sp);
        p.r = p.q == 0 || a.m.R == 1 ? 0 : p.q / a.nkp;
        p.kc = p.q - p.r * a.nkp;
      };
      auto advance = [&](Pos& p) {
        if (++p.q == p.q1) {
          p.w.next(a);
          start(p);
        } else if (++p.kc == a.nkp) {
          p.kc = 0, ++p.r;
        }
      };
      auto scales = [&](const Pos& p, float (&s)[U::NS]) {
        if constexpr (FA::SC) units.scales(s, a.m.A.ks + p.r * a.m.A.ks_r + p.kc * kBK, (int)min(a.m.K - p.kc * kBK, (long long)kBK));
      };
      Pos cur{Walk(a), 0, 0, 0, 0};
      start(cur);
      if (group == 1) advance(cur);
      float sc[U::NS], scn[U::NS];
      if (cur.w.in(a)) scales(cur, sc);
      auto fitted = [&](float (&s)[U::NS]) {
        if constexpr (kFit) {
          norm::F<U::NS> f;
#pragma unroll
          for (int k = 0; k < U::NS; ++k) f.v[k] = s[k];
          f = norm::mul(f, norm::fill<U::NS>(down));
#pragma unroll
          for (int k = 0; k < U::NS; ++k) s[k] = f.v[k];
        }
      };
      fitted(sc);
      bool ok = true;
      for (int i = group; cur.w.in(a); i += kGroups) {
        Pos nxt = cur;
#pragma unroll
        for (int k = 0; k < kGroups; ++k) advance(nxt);
        if (nxt.w.in(a)) scales(nxt, scn);  // this group's next step's
        const int s = i % kStages, w = i % kRaws;
        uint4 v[U::N];
        ok = mbar_wait(&rawf[w], (i / kRaws) & 1, kWaitLimit);
        ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
        if (!ok) break;
        const uint4* src = reinterpret_cast<const uint4*>(raws + w * C::kSlot);
#pragma unroll
        for (int j = 0; j < U::N; ++j) v[j] = src[units.raw(j)];
        if (i >= kAs) ok = mbar_wait(&empty[(i - kAs) % kStages], ((i - kAs) / kStages) & 1, kWaitLimit);
        ok = __all_sync(0xffffffffu, ok) && !*abort_flag;
        if (!ok) break;
        __syncwarp();  // every lane has read its units
        if (lane == 0) mbar_arrive(&rawe[w]);
#pragma unroll
        for (int j = 0; j < U::N; ++j) units.template put<HALF>(v[j], j, sc, smem + i % kAs * kABytes);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[s]);
        cur = nxt;
#pragma unroll
        for (int k = 0; k < U::NS; ++k) sc[k] = scn[k];
        fitted(sc);
      }
      if (!ok) {
        i8_flag();
        *abort_flag = 1;
      }
    }
  } else if (warp == kTmaAWarp || warp == kTmaBWarp) {
    // ------------------------------------------------------------ TMA --
    auto copies = [&](auto which) {
      // A's integers go into the raw ring, 16-bit lines into the stage
      constexpr bool is_a = decltype(which)::value, ring = is_a && kRaw, km = is_a ? FA::KM : BKM;
      constexpr int slots = ring ? kRaws : kStages;
      const int lines = is_a ? kBM : km ? a.NB : (a.NB + 63) / 64 * 64;
      uint64_t *f = ring ? rawf : full, *e = ring ? rawe : empty;
      uint8_t* base = ring ? raws : is_a ? smem : bring;
      constexpr uint32_t pitch = ring ? C::kSlot : is_a ? kABytes : kBBytes, line = ring ? 64 : 128;
      const CUtensorMap* map = is_a ? &amap : &bmap;
      [[maybe_unused]] const long long I = is_a ? a.m.M : a.m.N;
      // a weight has one slice for all z
      const bool sliced = is_a ? a.m.A.z || a.m.A.r : a.m.B.z || a.m.B.r;
      int i = 0;
      bool ok = true;
      for (Walk c(a); c.in(a) && ok; c.next(a)) {
        const long long i0 = is_a ? c.m0() : c.n0(a), q0 = first_step(c.sp), q1 = last_step(c.sp);
        long long r = q0 == 0 || a.m.R == 1 ? 0 : q0 / a.nkp, kc = q0 - r * a.nkp;
        for (long long q = q0; q < q1; ++q, ++i, ++kc) {
          if (kc == a.nkp) kc = 0, ++r;
          const int s = i % slots;
          if ((i >= slots && !mbar_wait(&e[s], ((i / slots) - 1) & 1, kWaitLimit)) || *abort_flag) {
            ok = false;
            break;
          }
          const long long k0 = kc * kBK, zr = !sliced ? 0 : a.m.R == 1 ? c.z : r;
          uint8_t* d = base + s * pitch;
          tc_expect_tx(&f[s], lines * line);
          // boxes start inside the operand; past its ends the copy engine writes zeros
          if (!DISCO_IN_BOUNDS(i0 >= 0 && i0 < I && k0 >= 0 && k0 < a.m.K && zr >= 0 && zr < (long long)a.m.Z * a.m.R)) {
            mbar_complete_tx(&f[s], lines * line);
            continue;
          }
          if constexpr (km) {
            tc_tma_3d(d, map, (int)k0, (int)i0, (int)zr, &f[s]);
          } else {
            constexpr int wide = ring ? kBM : 64;  // m or n of a box
            for (int b = 0; b < lines / wide; ++b) tc_tma_3d(d + b * 64 * line, map, (int)i0 + wide * b, (int)k0, (int)zr, &f[s]);
          }
        }
      }
      if (!ok) {
        i8_flag();
        *abort_flag = 1;
        // the copies in flight end before the CTA does
        for (int back = 1; back <= slots && i - back >= 0; ++back)
          mbar_wait(&f[(i - back) % slots], ((i - back) / slots) & 1, 1u << 16);
      }
    };
    if (elected()) {
      if (warp == kTmaAWarp) copies(std::true_type());
      else copies(std::false_type());
    }
  } else if (warp == kMmaWarp) {
    // --------------------------------------------------------- MMA issuer --
    if (elected()) {
      const int nmma = (a.NB + 15) / 16 * 16;
      const uint32_t idesc = idesc_16_f32(kBM, nmma, HALF) | (FA::KM ? 0u : 1u << 15) | (BKM ? 0u : 1u << 16);
      int i = 0, tl = 0;
      bool ok = true;
      for (Walk c(a); c.in(a) && ok; c.next(a), ++tl) {
        const int ab = tl & (accs - 1), turn = tl / accs;
        const long long q0 = first_step(c.sp), q1 = last_step(c.sp);
        if (turn > 0 && !mbar_wait(&acce[ab], (turn - 1) & 1, kWaitLimit)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (long long q = q0; q < q1; ++q, ++i) {
          const int s = i % kStages;
          if (!mbar_wait(&full[s], (i / kStages) & 1, kWaitLimit) || *abort_flag) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + i % kAs * kABytes), sb = smem_u32(bring + s * kBBytes);
#pragma unroll
          for (int ks = 0; ks < kBK / 16; ++ks) {
            // 16 k: 32 bytes of every line (k contiguous), or 16 lines; boxes of 64 m or n are 8 KB apart
            const uint64_t ad = FA::KM ? tc_desc(sa + ks * 32, 16) : tc_desc(sa + ks * 2048, 8192);
            const uint64_t bd = BKM ? tc_desc(sb + ks * 32, 16) : tc_desc(sb + ks * 2048, 8192);
            umma_bf16(tmem + ab * acc_cols, ad, bd, idesc, (q > q0 || ks > 0) ? 1u : 0u);
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
    const int q4 = warp & 3;                    // TMEM lanes 32 q4 ..: m of this warp
    uint8_t* stg = staging + warp * C::kStaging;  // 16-byte piece s of row r at piece s ^ (r / 2 % 4): no bank conflicts
    float* cs = reinterpret_cast<float*>(colscale + warp * C::kCols);
    const bool split = a.part != nullptr, scaled = C::kCols && !split;
    [[maybe_unused]] const float up = kFit ? fit_up(*most) : 1.0f;
    const int type = split ? DISCO_F32 : a.out_type, eb = type == DISCO_F32 ? 4 : 2;
    const bool h16 = type == DISCO_F16;
    // chunks of 32 columns; where two warps share the lanes, every second chunk, or all of every second tile
    const int half = warp >> 2, c00 = turns ? 0 : half * 32, step = turns ? 32 : 8 * kEpiWarps;
    int tl = 0;
    Walk c(a);
    if (turns && half) c.next(a), ++tl;
    auto row_scale = [&](const Walk& w) {
      const long long row = w.m0() + q4 * 32 + lane;
      return scaled && w.in(a) && row < a.m.M ? __ldg(a.m.rs + w.z * a.m.rs_z + row) : 1.0f;
    };
    float rs, rs_next = row_scale(c);
    int cs_n = -1;  // the n tile whose scales are held
    while (c.in(a)) {
      const int ab = tl & (accs - 1);
      const long long row0 = c.m0() + q4 * 32, n0 = c.n0(a);
      Walk next = c;
      next.next(a);
      if (turns) next.next(a);
      rs = rs_next;
      rs_next = row_scale(next);  // a tile ahead
      if (scaled && cs_n != c.n) {
        for (int n = lane; n < a.NB; n += 32) cs[n] = n0 + n < a.m.N ? __ldg(a.m.cs + n0 + n) : 0.0f;
        cs_n = c.n;
        __syncwarp();
      }
      bool fin = mbar_wait(&accf[ab], (tl / accs) & 1, kWaitLimit);
      fin = __all_sync(0xffffffffu, fin) && !*abort_flag;
      if (!fin) {
        if (lane == 0) i8_flag();
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const int rows = (int)min(a.m.M - row0, 32LL);  // may be negative
      const int cols = (int)min(a.m.N - n0, (long long)a.NB);
      const long long slice = (c.sp * (long long)a.m.Z + c.z) * a.m.M * a.m.N;
      // first of this warp's outputs; rows of the output are n (TR) or m
      uint8_t* out = (uint8_t*)(split ? (void*)a.part : a.m.out) + (slice + (TR ? n0 * a.m.M + row0 : row0 * a.m.N + n0)) * eb;
      const long long pitch = (TR ? a.m.M : a.m.N) * eb;
      for (int c0 = c00; c0 < cols && rows > 0; c0 += step) {
        uint32_t v[32];
        tmem_ld32(tmem + ab * acc_cols + ((uint32_t)(q4 * 32) << 16) + c0, v);
        if constexpr (kFit)
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * up);
        if (scaled) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = *reinterpret_cast<const float4*>(cs + c0 + e);
            // the product of the scales may leave fp32's range where y does not
            const norm::F<4> sum{{__uint_as_float(v[e]), __uint_as_float(v[e + 1]), __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])}};
            const norm::F<4> x = norm::mul(norm::mul(sum, norm::F<4>{{f.x, f.y, f.z, f.w}}), norm::fill<4>(rs));
#pragma unroll
            for (int k = 0; k < 4; ++k) v[e + k] = __float_as_uint(x.v[k]);
          }
        }
        const int left = min(32, cols - c0);
        if constexpr (TR) {
          uint8_t* o = out + (long long)c0 * pitch;
          if (eb == 2 && a.vec) {
            // pairs of n of 32 m through shared memory, then 8 m of both n to a lane (2-byte
            // stores straight from the registers took 141 us instead of 71 for dx of 2 x 256 -> 128 channels)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              *reinterpret_cast<uint32_t*>(stg + (e / 2) * 128 + (lane ^ (e / 2 & 1) << 2) * 4) = pack2_16(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), h16);
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int pair = (lane >> 2) + 8 * h, seg = lane & 3;
              const uint8_t* row = stg + pair * 128;  // the 16-byte words of odd pairs are swapped: no bank conflicts
              const uint4 x = *reinterpret_cast<const uint4*>(row + ((2 * seg ^ (pair & 1)) << 4)), y = *reinterpret_cast<const uint4*>(row + (((2 * seg + 1) ^ (pair & 1)) << 4));
              if (seg * 8 < rows) {
                uint8_t* d = o + 2 * pair * pitch + seg * 16;
                if (2 * pair < left)
                  *reinterpret_cast<uint4*>(d) = make_uint4(__byte_perm(x.x, x.y, 0x5410), __byte_perm(x.z, x.w, 0x5410),
                                                            __byte_perm(y.x, y.y, 0x5410), __byte_perm(y.z, y.w, 0x5410));
                if (2 * pair + 1 < left)
                  *reinterpret_cast<uint4*>(d + pitch) = make_uint4(__byte_perm(x.x, x.y, 0x7632), __byte_perm(x.z, x.w, 0x7632),
                                                                    __byte_perm(y.x, y.y, 0x7632), __byte_perm(y.z, y.w, 0x7632));
              }
            }
            __syncwarp();
          } else if (lane < rows) {  // the warp's lanes are neighbours in memory
            o += lane * eb;
            if (type == DISCO_F32) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                if (e < left) *reinterpret_cast<uint32_t*>(o) = v[e];
                next_row(o, pitch);
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const uint32_t two = pack2_16(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), h16);
                if (e < left) *reinterpret_cast<uint16_t*>(o) = (uint16_t)two;
                next_row(o, pitch);
                if (e + 1 < left) *reinterpret_cast<uint16_t*>(o) = (uint16_t)(two >> 16);
                next_row(o, pitch);
              }
            }
          }
        } else {
          // 64 bytes of each of the warp's 32 rows at a time through shared memory
          auto emit = [&](int w0, int n) {  // n columns from c0 + w0 are staged
            __syncwarp();
            const int some = min(n, left - w0);
            uint8_t* o = out + (long long)(c0 + w0) * eb;
            if (a.vec) {
#pragma unroll
              for (int h = 0; h < 4; ++h) {
                const int idx = lane + 32 * h, row = idx >> 2, seg = idx & 3;
                if (row < rows && seg * 16 < some * eb)
                  *reinterpret_cast<uint4*>(o + row * pitch + seg * 16) = *reinterpret_cast<const uint4*>(stg + row * 64 + ((seg ^ (row >> 1)) & 3) * 16);
              }
            } else {
              const int step = 64 / eb, col = lane & (step - 1);  // 32 lanes over one row of 2-byte or two of 4-byte elements
              if (col < some)
#pragma unroll 4
                for (int row = lane / step; row < rows; row += 32 / step) {
                  const uint8_t* s = stg + row * 64 + (((col * eb >> 4) ^ (row >> 1)) & 3) * 16 + (col * eb & 15);
                  if (eb == 2) *reinterpret_cast<uint16_t*>(o + row * pitch + col * 2) = *reinterpret_cast<const uint16_t*>(s);
                  else *reinterpret_cast<uint32_t*>(o + row * pitch + col * 4) = *reinterpret_cast<const uint32_t*>(s);
                }
            }
            __syncwarp();
          };
          auto stage = [&](int g, uint4 x) { *reinterpret_cast<uint4*>(stg + lane * 64 + ((g ^ (lane >> 1)) & 3) * 16) = x; };
          if (type == DISCO_F32) {
#pragma unroll
            for (int g = 0; g < 4; ++g) stage(g, make_uint4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]));
            emit(0, 16);
            if (left > 16) {
#pragma unroll
              for (int g = 0; g < 4; ++g) stage(g, make_uint4(v[16 + 4 * g], v[17 + 4 * g], v[18 + 4 * g], v[19 + 4 * g]));
              emit(16, 16);
            }
          } else {
            auto two = [&](int e) { return pack2_16(__uint_as_float(v[e]), __uint_as_float(v[e + 1]), h16); };
#pragma unroll
            for (int g = 0; g < 4; ++g) stage(g, make_uint4(two(8 * g), two(8 * g + 2), two(8 * g + 4), two(8 * g + 6)));
            emit(0, 32);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acce[ab]);
      c = next;
      tl += turns ? 2 : 1;
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

// `lines` of 64 elements to a copy: of 64 k, or (MN-major) 64 of them, of 64 m or n (integers: 128).
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
  const int es = o.bits / 8;
  const long long slice = max(o.z, o.r);
  const cuuint64_t dims[3] = {(cuuint64_t)(o.k_major ? K : I), (cuuint64_t)(o.k_major ? I : K), (cuuint64_t)(slice ? ZR : 1)};
  const cuuint64_t strides[2] = {(cuuint64_t)o.ld * es, (cuuint64_t)(slice ? slice : o.ld * dims[1]) * es};
  const cuuint32_t box[3] = {o.k_major || es == 2 ? 64u : (cuuint32_t)kBM, (cuuint32_t)(o.k_major ? lines : 64), 1}, estr[3] = {1, 1, 1};
  const CUtensorMapDataType type = es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                           : f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const CUresult cr = enc(map, type, 3, const_cast<void*>(o.p), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          es == 1 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (cr != CUDA_SUCCESS) return fail(DISCO_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)cr);
  return DISCO_OK;
}

template <class FA, bool BKM, bool HALF, bool TR>
int tc_launch(const TcArgs& a, cudaStream_t st) {
  CUtensorMap amap = {}, bmap = {};
  int rc;
  if ((rc = tc_encode(&amap, a.m.A, a.m.M, a.m.K, a.m.Z * a.m.R, kBM, HALF))) return rc;
  if ((rc = tc_encode(&bmap, a.m.B, a.m.N, a.m.K, a.m.Z * a.m.R, a.NB, HALF))) return rc;
  constexpr size_t kSmem = Plan<FA>::kSmem;
  auto kern = i8_tc_kernel<FA, BKM, HALF, TR>;
  return norm::launch(kern, (int)min(a.tiles, (uint32_t)kSMs), Plan<FA>::kThreads, 1, a.after, kSmem, kSmem, st, "i8_tc_kernel", amap, bmap, a);
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
