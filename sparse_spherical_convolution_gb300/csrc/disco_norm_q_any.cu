// disco_norm_q_any.cu -- tile kernels of the channel norm with its 8-bit copy, any
// group size.

#include "disco_norm_tile.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_q_any_bounds)

namespace norm {

int norm_q_any_by_tiles(const NormArgs& a, const Tiling& g, disco_dtype dtype, cudaStream_t st) {
  const int ng_max = min(a.NG, (g.cpc + a.G - 1) / a.G + 1);
  int rc = DISCO_OK;
#define CALL(T) rc = norm_tile<kAtomicQ, T>(a, g, ng_max, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

}  // namespace norm
}  // namespace disco
