// disco_i8_dx.cu -- the activation's gradient of the integer product on the tensor
// cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_dx_bounds)
DISCO_I8_STATUS_READER(i8_dx_status)

namespace i8 {

int tc_dx(const TcArgs& a, cudaStream_t st) {
  using Rows = Form<2, true, 0>;
  using Grid = Form<2, false, 0>;
  if (a.m.A.k_major) return a.m.f16 ? tc_launch<Rows, false, true, false>(a, st) : tc_launch<Rows, false, false, false>(a, st);
  return a.m.f16 ? tc_launch<Grid, false, true, true>(a, st) : tc_launch<Grid, false, false, true>(a, st);
}

}  // namespace i8
}  // namespace disco
