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

// out[z][m][n] = rs[m] cs[z cs_z + n] sum_{r < R, k < K} A(m, k) B(n, k); rs and cs may be null.
struct MmArgs {
  Operand A, B;
  const float *rs, *cs;
  void* out;
  long long cs_z, M, N, K;
  int Z, R, f16;
};

}  // namespace i8
}  // namespace disco
