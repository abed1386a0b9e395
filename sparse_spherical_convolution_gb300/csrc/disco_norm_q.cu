// disco_norm_q.cu -- tile kernels of the channel norm with its 8-bit copy, groups
// that a thread's channels and a CTA do not straddle.

#include "disco_norm_tile.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_q_bounds)

namespace norm {

int norm_q_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st) {
  Tiling g;
  if (!plan_tiles(a.B, a.C, a.P, elem_bytes(dtype), true, &g)) return DISCO_ERR_UNSUPPORTED;
  // a block of `apart` threads holds apart * NCH neighbouring channels
  const bool rows = (a.NG == 1 || a.G % (g.apart * g.NCH) == 0) && (g.CL == 1 || g.cpc % a.G == 0);
  if (!rows) return norm_q_any_by_tiles(a, g, dtype, st);
  const int ng_max = min(a.NG, (g.cpc + a.G - 1) / a.G);
  int rc = DISCO_OK;
#define CALL(T) rc = norm_tile<kRowsQ, T>(a, g, ng_max, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

}  // namespace norm
}  // namespace disco
