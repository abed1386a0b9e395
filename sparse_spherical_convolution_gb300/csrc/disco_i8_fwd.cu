// disco_i8_fwd.cu -- the integer product on the tensor cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_fwd_bounds)
DISCO_I8_STATUS_READER(i8_fwd_status)

namespace i8 {

int tc_fwd(const TcArgs& a, cudaStream_t st) {
  if (!a.m.A.k_major) return tc_launch<Form<1, false, 0>, true, true, true>(a, st);  // grids
  if (a.m.transposed) return tc_launch<Form<1, true, 0>, true, true, true>(a, st);   // rows, A the weight
  return tc_launch<Form<1, true, 0>, true, true, false>(a, st);
}

}  // namespace i8
}  // namespace disco
