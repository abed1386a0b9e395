// disco_tokens_grid.cu -- grids of tokens by tiles whose rows are whole words (disco_tokens.cuh).

#include "disco_tokens.cuh"

namespace disco {

DISCO_BOUNDS_READER(tokens_grid_bounds)

namespace i8 {

int tokens_grid(const TokenArgs& a, bool glu, disco_dtype dtype, cudaStream_t st) {
  int rc;
#define CALL(T) rc = tiles_of<T, false>(a, glu, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

}  // namespace i8
}  // namespace disco
