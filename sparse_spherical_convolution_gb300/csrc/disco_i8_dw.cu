// disco_i8_dw.cu -- the weight's gradient of the integer product on the tensor
// cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_dw_bounds)
DISCO_I8_STATUS_READER(i8_dw_status)

namespace i8 {

template <bool HALF, bool KM>
int dw(const TcArgs& a, cudaStream_t st) {
  using F = Form<1, KM, 1>;
  if (a.ala && a.alb) return tc_launch<F, KM, HALF, true, true, true>(a, st);
  return a.alb ? tc_launch<F, KM, HALF, false, true, true>(a, st) : tc_launch<F, KM, HALF, false, false, true>(a, st);
}

int tc_dw(const TcArgs& a, cudaStream_t st) {
  if (a.m.f16) return a.m.A.k_major ? dw<true, true>(a, st) : dw<true, false>(a, st);
  return a.m.A.k_major ? dw<false, true>(a, st) : dw<false, false>(a, st);
}

}  // namespace i8
}  // namespace disco
