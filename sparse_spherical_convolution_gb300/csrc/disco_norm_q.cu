// disco_norm_q.cu -- tile kernels of the channel norm with its 8-bit copy.

#include "disco_norm_tile.cuh"

namespace disco {

DISCO_BOUNDS_READER(norm_q_bounds)

namespace norm {

int norm_q_by_tiles(const NormArgs& a, disco_dtype dtype, cudaStream_t st) {
  Tiling g;
  if (!plan_tiles(a.B, a.C, a.P, elem_bytes(dtype), true, &g)) return DISCO_ERR_UNSUPPORTED;
  // rows: a thread's channels lie in one group, a group in one CTA
  const bool rows = (a.NG == 1 || a.G % g.NCH == 0) && (g.CL == 1 || g.cpc % a.G == 0);
  const int ng_max = min(a.NG, (g.cpc + a.G - 1) / a.G + (rows ? 0 : 1));
  int rc = DISCO_OK;
#define CALL(T) rc = rows ? norm_tile<kRowsQ, T>(a, g, ng_max, st) : norm_tile<kAtomicQ, T>(a, g, ng_max, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

}  // namespace norm
}  // namespace disco
