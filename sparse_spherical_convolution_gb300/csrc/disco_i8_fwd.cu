// disco_i8_fwd.cu -- the integer product on the tensor cores (disco_i8_tc.cuh).

#include "disco_i8_tc.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_fwd_bounds)
DISCO_I8_STATUS_READER(i8_fwd_status)

namespace i8 {

int tc_fwd(const TcArgs& a, bool aligned, cudaStream_t st) {
  using K8 = Form<1, true, 0>;
  using N8 = Form<1, false, 0>;
  if (a.m.B.k_major) return aligned ? tc_launch<K8, K8, true, true>(a, st) : tc_launch<K8, K8, true, false>(a, st);
  return aligned ? tc_launch<K8, N8, true, true>(a, st) : tc_launch<K8, N8, true, false>(a, st);
}

}  // namespace i8
}  // namespace disco
