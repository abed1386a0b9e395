// disco_i8_fwd.cu -- the integer product on the tensor cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_fwd_bounds)
DISCO_I8_STATUS_READER(i8_fwd_status)

namespace i8 {

int tc_fwd(const TcArgs& a, cudaStream_t st) {
  using Rows = Form<1, true, 0>;
  using Grid = Form<1, false, 0>;
  if (a.m.A.k_major && a.m.transposed)  // rows, A the weight
    return a.ala ? tc_launch<Rows, true, true, true, true, true>(a, st) : tc_launch<Rows, true, true, false, true, true>(a, st);
  if (a.m.A.k_major) return a.ala ? tc_launch<Rows, true, true, true, true, false>(a, st) : tc_launch<Rows, true, true, false, true, false>(a, st);
  return a.ala ? tc_launch<Grid, true, true, true, true, true>(a, st) : tc_launch<Grid, true, true, false, true, true>(a, st);
}

}  // namespace i8
}  // namespace disco
