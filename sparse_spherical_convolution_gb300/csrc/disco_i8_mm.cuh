// disco_i8_mm.cuh -- how the integer products and their gradients are described
// to the kernels.  Not part of the ABI.
#pragma once

#include "disco_i8.cuh"

namespace disco {
namespace i8 {

// One operand X(i, k), i = m or n: element z Z + r R + (k_major ? i ld + k : k ld + i)
// of `p`, for output slice z and reduction slice r, times ks[r ks_r + k] where given.
struct Operand {
  const void* p;
  const float* ks;
  long long z, r, ld, ks_r;
  int bits;  // 8: integers, 16: fp16 or bf16
  bool k_major;
};

// The power of two that is taken out of the scales of an fp16 gradient before scale * integer is rounded
// to fp16: with it the largest finite scale lies in [128, 256), so no term overflows, and small scales keep
// their digits down to 2^-21 of the largest.  (Without it weights below 1e-5 lost digits to fp16's
// subnormals, and scales above 516 became infinite.)
struct Range {
  const float* v;  // n values with the largest magnitude of the scales: the scales, or the largest of parts of them; null: scales as they are
  int n;
};
// The bits of a block's share of the largest finite |v|; all lanes of a warp call it, the i-th of `step` threads.
__device__ __forceinline__ uint32_t largest(const float* v, long long n, long long i, long long step) {
  uint32_t m = 0;
  auto add = [&](float f) {
    const uint32_t b = __float_as_uint(f) & 0x7fffffffu;
    if (b < 0x7f800000u) m = max(m, b);
  };
  const long long words = n / 4;
  if (i < n - 4 * words) add(__ldcg(v + 4 * words + i));
  for (; i < words; i += step) {
    const float4 f = __ldcg(reinterpret_cast<const float4*>(v) + i);
    add(f.x), add(f.y), add(f.z), add(f.w);
  }
  return __reduce_max_sync(0xffffffffu, m);
}
// What a scale is multiplied by, and what a sum of terms is, from the bits of the largest
// scale; both are normal numbers.
__device__ __forceinline__ int fit(uint32_t most) { return max((int)(most >> 23), 14); }
__device__ __forceinline__ float fit_down(uint32_t most) { return __uint_as_float((uint32_t)(261 - fit(most)) << 23); }
__device__ __forceinline__ float fit_up(uint32_t most) { return __uint_as_float((uint32_t)(fit(most) - 7) << 23); }

// out[z][m][n] = rs[z rs_z + m] cs[n] sum_{r < R, k < K} A(m, k) B(n, k), or with
// `transposed` out[z][n][m]; rs and cs may both be null.
struct MmArgs {
  Operand A, B;
  const float *rs, *cs;
  void* out;
  long long rs_z, M, N, K;
  int Z, R, f16;
  bool transposed;
  Range range;  // of A's ks, or of the scales that B's integers were multiplied by
};

// The steps (of 64 k) of one sum in an accumulator, at most.  The tensor cores cut off what a sum's
// 24 bits do not hold at each of the four instructions of a step, so a sum of one sign comes out too small: over 2
// million tokens by 1.7e-3 of it, three times fp16's rounding.  2048 instructions lose 2.4e-4 of a sum
// at a unit of 2^-23 each, and some 4e-5 where terms are alike and the sum grows evenly; and a wait for a
// part's sums stays short.  Parts are joined in fp32 with rounding to nearest.  Times with and without:
// dW of 400000 rows of 2048 by 1280 1.72 ms (3.04: its parts fill the SMs), 20 x 64 -> 64 on 360x720 320 us (307).
constexpr long long kPartSteps = 512;

// How the tensor-core kernel cuts a product (disco_i8_tc.cuh): tiles of 128 m x NB n
// of each z, their reduction of `steps` chunks of 64 k in nsplit parts.
struct TcArgs {
  MmArgs m;
  float* part;                 // fp32 sums of the parts, each laid out as out, or null
  int NB, nsplit, out_type, vec;        // vec: rows of what it writes start on 16 bytes
  bool after;                           // the launch before it wrote operands: begin while that one ends
  uint32_t mt, nt, tiles;               // of a z, of the call (with parts); below 2^31
  long long nkp, steps;                 // 64-k chunks of a slice r, of all
};

int tc_fwd(const TcArgs& a, cudaStream_t st);
int tc_dx(const TcArgs& a, cudaStream_t st);
int tc_dw(const TcArgs& a, cudaStream_t st);

}  // namespace i8
}  // namespace disco
