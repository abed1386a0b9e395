// disco_i8_dw.cu -- the weight's gradient of the integer product on the tensor
// cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_dw_bounds)
DISCO_I8_STATUS_READER(i8_dw_status)

namespace i8 {

template <bool HALF, bool ALN>
int dw(const TcArgs& a, cudaStream_t st) {
  if (a.m.A.k_major) return tc_launch<Form<2, true, 0>, Form<1, true, 1>, HALF, ALN>(a, st);
  return tc_launch<Form<2, false, 0>, Form<1, false, 1>, HALF, ALN>(a, st);  // rows
}

int tc_dw(const TcArgs& a, bool aligned, cudaStream_t st) {
  if (a.m.f16) return aligned ? dw<true, true>(a, st) : dw<true, false>(a, st);
  return aligned ? dw<false, true>(a, st) : dw<false, false>(a, st);
}

}  // namespace i8
}  // namespace disco
