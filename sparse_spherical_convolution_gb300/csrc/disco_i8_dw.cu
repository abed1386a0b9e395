// disco_i8_dw.cu -- the weight's gradient of the integer product on the tensor
// cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_dw_bounds)
DISCO_I8_STATUS_READER(i8_dw_status)

namespace i8 {

int tc_dw(const TcArgs& a, cudaStream_t st) {
  using Grid = Form<1, true, 1>;
  using Rows = Form<1, false, 1>;
  if (a.m.A.k_major) return a.m.f16 ? tc_launch<Grid, true, true, true>(a, st) : tc_launch<Grid, true, false, true>(a, st);
  return a.m.f16 ? tc_launch<Rows, false, true, true>(a, st) : tc_launch<Rows, false, false, true>(a, st);
}

}  // namespace i8
}  // namespace disco
