// disco_i8_dx.cu -- the activation's gradient of the integer product on the tensor
// cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_dx_bounds)
DISCO_I8_STATUS_READER(i8_dx_status)

namespace i8 {

template <bool HALF>
int dx(const TcArgs& a, cudaStream_t st) {
  using Rows = Form<2, true, 0>;
  using Grid = Form<2, false, 0>;
  if (a.m.A.k_major) return a.ala ? tc_launch<Rows, false, HALF, true, true, false>(a, st) : tc_launch<Rows, false, HALF, false, true, false>(a, st);
  return a.ala ? tc_launch<Grid, false, HALF, true, true, true>(a, st) : tc_launch<Grid, false, HALF, false, true, true>(a, st);
}

int tc_dx(const TcArgs& a, cudaStream_t st) { return a.m.f16 ? dx<true>(a, st) : dx<false>(a, st); }

}  // namespace i8
}  // namespace disco
