// disco_tokens_rows.cu -- tokens held in registers: rows, and single pixels of grids (disco_tokens.cuh).

#include "disco_tokens.cuh"

namespace disco {

DISCO_BOUNDS_READER(tokens_rows_bounds)

namespace i8 {

namespace {

// J words to a thread: few while the channels fit the threads (many CTAs to an SM), else more.
template <typename T, int V, int J, bool GLU, bool XQ, bool YQ>
int held(const TokenArgs& a, cudaStream_t st) {
  const int rc = held_as<T, V, J, GLU, XQ, YQ>(a, st);
  return rc != DISCO_ERR_UNSUPPORTED ? rc : held_as<T, V, 2 * J, GLU, XQ, YQ>(a, st);
}
template <typename T, int V>
int held(const TokenArgs& a, bool glu, cudaStream_t st) {
  if (!glu) return held<T, V, V == 1 ? 16 : 8, false, true, false>(a, st);
  constexpr int J = 4;
  if (a.xq && a.q) return held<T, V, J, true, true, true>(a, st);
  if (a.xq) return held<T, V, J, true, true, false>(a, st);
  if (a.q) return held<T, V, J, true, false, true>(a, st);
  return held_as<T, V, 4, true, false, false>(a, st);
}

}  // namespace

int tokens_held(const TokenArgs& a, bool glu, disco_dtype dtype, cudaStream_t st) {
  int rc;
#define CALL(T) rc = a.P == 1 && a.C % (16 / (int)sizeof(T)) == 0 ? held<T, 16 / (int)sizeof(T)>(a, glu, st) : held<T, 1>(a, glu, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

}  // namespace i8
}  // namespace disco
