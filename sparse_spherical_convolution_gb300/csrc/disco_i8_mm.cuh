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

// out[z][m][n] = rs[z rs_z + m] cs[n] sum_{r < R, k < K} A(m, k) B(n, k), or with
// `transposed` out[z][n][m]; rs and cs may both be null.
struct MmArgs {
  Operand A, B;
  const float *rs, *cs;
  void* out;
  long long rs_z, M, N, K;
  int Z, R, f16;
  bool transposed;
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
