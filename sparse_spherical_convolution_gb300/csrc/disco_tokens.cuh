// disco_tokens.cuh -- arguments of the kernels that work token by token
// (disco_tokens.cu).  Not part of the ABI.
#pragma once

#include "disco_i8.cuh"

namespace disco {
namespace i8 {

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

}  // namespace i8
}  // namespace disco
