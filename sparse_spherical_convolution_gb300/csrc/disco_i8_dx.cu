// disco_i8_dx.cu -- the activation's gradient of the integer product on the tensor
// cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_dx_bounds)
DISCO_I8_STATUS_READER(i8_dx_status)

namespace i8 {

template <bool HALF, bool ALN>
int dx(const TcArgs& a, cudaStream_t st) {
  if (a.m.A.bits == 16) return tc_launch<Form<2, true, 0>, Form<1, false, 1>, HALF, ALN>(a, st);  // rows
  return tc_launch<Form<1, false, 1>, Form<2, false, 0>, HALF, ALN>(a, st);
}

int tc_dx(const TcArgs& a, bool aligned, cudaStream_t st) {
  if (a.m.f16) return aligned ? dx<true, true>(a, st) : dx<true, false>(a, st);
  return aligned ? dx<false, true>(a, st) : dx<false, false>(a, st);
}

}  // namespace i8
}  // namespace disco
