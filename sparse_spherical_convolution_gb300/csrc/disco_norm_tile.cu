// disco_norm_tile.cu -- tile kernels of the channel norm without the 8-bit copy.

#include "disco_norm_tile.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_tile_bounds)

namespace norm {

int norm_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st) {
  Tiling g;
  if (!plan_tiles(a.B, a.C, a.P, elem_bytes(dtype), true, &g)) return DISCO_ERR_UNSUPPORTED;
  int rc = DISCO_OK;
#define CALL(T) rc = norm_tile<kNoQ, T>(a, g, 0, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

}  // namespace norm
}  // namespace disco
