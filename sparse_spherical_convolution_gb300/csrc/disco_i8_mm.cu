// disco_i8_mm.cu -- products over the channels of each token with activations and
// weights in 8-bit integers, and their gradients from the 8-bit activation:
// checks, the choice of a kernel, and the general one.
//
//   y[b,o,p]  = scale[b,p] wscale[o] sum_c W[o,c] q[b,c,p]      (disco_matmul_i8)
//   dx[b,c,p] = sum_o wscale[o] W[o,c] dy[b,o,p]                (disco_matmul_i8_bwd_input)
//   dW[o,c]   = sum_{b,p} dy[b,o,p] scale[b,p] q[b,c,p]         (disco_matmul_i8_bwd_weight)
//
// Each is out[z][m][n] = rs[m] cs[n] sum_k ks[k] A(m, k) B(n, k), row-major with n
// the contiguous direction of the output: pixels (grids) or channels (rows).

#include "disco_i8_mm.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_mm_bounds)

namespace {

using namespace i8;

constexpr int kAnyThreads = 256;

// The parts' sums in their order, scaled and rounded.
template <typename TO>
__global__ void __launch_bounds__(kAnyThreads) mm_join_kernel(const MmArgs a, const float* part, int nsplit, long long n) {
  for (long long i = (long long)blockIdx.x * kAnyThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kAnyThreads) {
    float v = 0.0f;
    for (int s = 0; s < nsplit; ++s) v += part[s * n + i];
    const long long r = i / a.N, c = i - r * a.N;
    if (a.cs) v *= a.cs[r / a.M * a.cs_z + c];
    if (a.rs) v *= a.rs[r % a.M];
    ((TO*)a.out)[i] = from_f32<TO>(v);
  }
}

// The cut of a product by its sizes alone (the workspace's bytes follow from it).
// Tiles of 256 n; where they do not fill the SMs, the reduction is split into
// parts of 8 steps at least, and where that leaves half of the SMs idle, tiles get narrower.
struct Cut {
  int NB, nsplit;
  long long mt, nt, nkp, steps;
  Cut(long long M, long long N, long long K, int Z, int R) {
    mt = (M + 127) / 128;
    nkp = (K + 63) / 64;
    steps = nkp * R;
    NB = N >= 256 ? 256 : (int)((N + 63) / 64 * 64);
    for (;;) {
      nt = (N + NB - 1) / NB;
      const long long tiles = mt * nt * Z;
      nsplit = (int)max(1LL, min(steps / 8, kSMs / tiles));
      if (tiles * nsplit >= kSMs / 2 || NB == 64) break;
      NB = NB > 128 ? 128 : 64;
    }
  }
  size_t bytes(long long M, long long N, int Z) const { return nsplit > 1 ? (size_t)nsplit * Z * M * N * 4 : 16; }
};

bool rows_aligned(const Operand& o) {
  const int es = o.bits / 8;
  return o.ld * es % 16 == 0 && o.z * es % 16 == 0 && o.r * es % 16 == 0;
}

int run(const MmArgs& m, disco_dtype dtype, void* ws, int (*tc)(const TcArgs&, bool, cudaStream_t), cudaStream_t st) {
  const Cut c(m.M, m.N, m.K, m.Z, m.R);
  TcArgs a = {};
  a.m = m;
  a.enda = (const uint8_t*)m.A.p + m.A.n * (m.A.bits / 8);
  a.endb = (const uint8_t*)m.B.p + m.B.n * (m.B.bits / 8);
  a.NB = c.NB, a.nsplit = c.nsplit, a.mt = c.mt, a.nt = c.nt, a.nkp = c.nkp, a.steps = c.steps;
  a.part = c.nsplit > 1 ? (float*)ws : nullptr;
  a.out_type = dtype;
  a.vec = m.N * (a.part ? 4 : elem_bytes(dtype)) % 16 == 0;
  a.tiles = c.mt * c.nt * m.Z * c.nsplit;
  // the copy engine's coordinates are 32-bit
  const bool aligned = rows_aligned(m.A) && rows_aligned(m.B) && max(max(m.M, m.N), m.K) < 1LL << 31 && max(m.A.n, m.B.n) < 1LL << 38;
  int rc = tc(a, aligned, st);
  if (rc || !a.part) return rc;
  const long long n = m.Z * m.M * m.N;
  const int grid = (int)min((n + kAnyThreads - 1) / kAnyThreads, (long long)kSMs * 8);
#define CALL(T) mm_join_kernel<T><<<grid, kAnyThreads, 0, st>>>(m, a.part, c.nsplit, n)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("mm_join_kernel");
}

// Sizes of a product; 16-bit types only for the gradients.
int check_mm(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype, bool grad) {
  int rc;
  if ((rc = check_shape(B, Cin, P, dtype)) || (rc = check_shape(B, Cout, P, dtype))) return rc;
  if (grad && dtype == DISCO_F32) return fail(DISCO_ERR_UNSUPPORTED, "gradients take bf16 or fp16");
  if ((double)Cin * Cout > 1e12) return fail(DISCO_ERR_UNSUPPORTED, "more than 1e12 weights");
  return DISCO_OK;
}

// The workspace as a buffer that overlaps nothing.
int check_ws(const void* ws, size_t have, size_t need) {
  if (have < need || (need && !ws)) return fail(DISCO_ERR_WORKSPACE, "workspace of %zu bytes, the call needs %zu", have, need);
  return DISCO_OK;
}

}  // namespace
}  // namespace disco

using namespace disco;
using namespace disco::i8;

extern "C" size_t disco_matmul_i8_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, false)) return 0;
  return P == 1 ? Cut(B, Cout, Cin, 1, 1).bytes(B, Cout, 1) : Cut(Cout, P, Cin, B, 1).bytes(Cout, P, B);
}

extern "C" size_t disco_matmul_i8_bwd_input_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return P == 1 ? Cut(B, Cin, Cout, 1, 1).bytes(B, Cin, 1) : Cut(Cin, P, Cout, B, 1).bytes(Cin, P, B);
}

extern "C" size_t disco_matmul_i8_bwd_weight_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return P == 1 ? Cut(Cout, Cin, B, 1, 1).bytes(Cout, Cin, 1) : Cut(Cout, Cin, P, 1, B).bytes(Cout, Cin, 1);
}

extern "C" int disco_matmul_i8(const void* q, const float* scale, const void* W, const float* wscale, void* y, int32_t B,
                               int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype, void* workspace, size_t workspace_bytes,
                               void* stream) {
  disco::NvtxScope nvtx_scope("disco_matmul_i8");
  int rc;
  if ((rc = check_mm(B, Cin, Cout, P, dtype, false))) return rc;
  if (!q || !scale || !W || !wscale || !y) return fail(DISCO_ERR_INVALID_ARG, "q, scale, W, wscale or y is null");
  const size_t need = disco_matmul_i8_workspace_bytes(B, Cin, Cout, P, dtype);
  if ((rc = check_ws(workspace, workspace_bytes, need)) || (rc = check_device())) return rc;
  const size_t T = (size_t)B * P, w = (size_t)Cout * Cin;
  const Buffer in[] = {{q, T * Cin, "q"}, {scale, T * 4, "scale"}, {W, w, "W"}, {wscale, (size_t)Cout * 4, "wscale"}};
  const Buffer out[] = {{y, T * Cout * elem_bytes(dtype), "y"}, {workspace, need, "workspace"}};
  const unsigned in_place[] = {0, 0, 0, 0};
  if ((rc = check_buffers(in, in_place, 4, out, 2))) return rc;
  MmArgs a = {};
  a.out = y;
  a.K = Cin;
  a.R = 1;
  if (P == 1) {  // rows: m = token, n = output channel
    a.A = {q, nullptr, 0, 0, Cin, 0, 8, true, (long long)T * Cin};
    a.B = {W, nullptr, 0, 0, Cin, 0, 8, true, (long long)w};
    a.rs = scale, a.cs = wscale;
    a.M = B, a.N = Cout, a.Z = 1;
  } else {  // m = output channel, n = pixel
    a.A = {W, nullptr, 0, 0, Cin, 0, 8, true, (long long)w};
    a.B = {q, nullptr, Cin * P, 0, P, 0, 8, false, (long long)T * Cin};
    a.rs = wscale, a.cs = scale, a.cs_z = P;
    a.M = Cout, a.N = P, a.Z = B;
  }
  return run(a, dtype, workspace, tc_fwd, (cudaStream_t)stream);
}

extern "C" int disco_matmul_i8_bwd_input(const void* dy, const void* W, const float* wscale, void* dx, int32_t B, int32_t Cin,
                                         int32_t Cout, int64_t P, disco_dtype dtype, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  disco::NvtxScope nvtx_scope("disco_matmul_i8_bwd_input");
  int rc;
  if ((rc = check_mm(B, Cin, Cout, P, dtype, true))) return rc;
  if (!dy || !W || !wscale || !dx) return fail(DISCO_ERR_INVALID_ARG, "dy, W, wscale or dx is null");
  const size_t need = disco_matmul_i8_bwd_input_workspace_bytes(B, Cin, Cout, P, dtype);
  if ((rc = check_ws(workspace, workspace_bytes, need)) || (rc = check_device())) return rc;
  const size_t T = (size_t)B * P, w = (size_t)Cout * Cin;
  const Buffer in[] = {{dy, T * Cout * 2, "dy"}, {W, w, "W"}, {wscale, (size_t)Cout * 4, "wscale"}};
  const Buffer out[] = {{dx, T * Cin * 2, "dx"}, {workspace, need, "workspace"}};
  const unsigned in_place[] = {0, 0, 0};
  if ((rc = check_buffers(in, in_place, 3, out, 2))) return rc;
  MmArgs a = {};
  a.out = dx;
  a.f16 = dtype == DISCO_F16;
  a.K = Cout;
  a.R = 1;
  if (P == 1) {  // m = token, n = input channel
    a.A = {dy, nullptr, 0, 0, Cout, 0, 16, true, (long long)T * Cout};
    a.B = {W, wscale, 0, 0, Cin, 0, 8, false, (long long)w};
    a.M = B, a.N = Cin, a.Z = 1;
  } else {  // m = input channel, n = pixel
    a.A = {W, wscale, 0, 0, Cin, 0, 8, false, (long long)w};
    a.B = {dy, nullptr, Cout * P, 0, P, 0, 16, false, (long long)T * Cout};
    a.M = Cin, a.N = P, a.Z = B;
  }
  return run(a, dtype, workspace, tc_dx, (cudaStream_t)stream);
}

extern "C" int disco_matmul_i8_bwd_weight(const void* dy, const void* q, const float* scale, void* dW, int32_t B, int32_t Cin,
                                          int32_t Cout, int64_t P, disco_dtype dtype, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  disco::NvtxScope nvtx_scope("disco_matmul_i8_bwd_weight");
  int rc;
  if ((rc = check_mm(B, Cin, Cout, P, dtype, true))) return rc;
  if (!dy || !q || !scale || !dW) return fail(DISCO_ERR_INVALID_ARG, "dy, q, scale or dW is null");
  const size_t need = disco_matmul_i8_bwd_weight_workspace_bytes(B, Cin, Cout, P, dtype);
  if ((rc = check_ws(workspace, workspace_bytes, need)) || (rc = check_device())) return rc;
  const size_t T = (size_t)B * P;
  const Buffer in[] = {{dy, T * Cout * 2, "dy"}, {q, T * Cin, "q"}, {scale, T * 4, "scale"}};
  const Buffer out[] = {{dW, (size_t)Cout * Cin * 2, "dW"}, {workspace, need, "workspace"}};
  const unsigned in_place[] = {0, 0, 0};
  if ((rc = check_buffers(in, in_place, 3, out, 2))) return rc;
  MmArgs a = {};
  a.out = dW;
  a.f16 = dtype == DISCO_F16;
  a.M = Cout, a.N = Cin, a.Z = 1;
  if (P == 1) {  // k = token
    a.A = {dy, nullptr, 0, 0, Cout, 0, 16, false, (long long)T * Cout};
    a.B = {q, scale, 0, 0, Cin, 0, 8, false, (long long)T * Cin};
    a.K = B, a.R = 1;
  } else {  // k = pixel, summed over the samples too
    a.A = {dy, nullptr, 0, Cout * P, P, 0, 16, true, (long long)T * Cout};
    a.B = {q, scale, 0, Cin * P, P, P, 8, true, (long long)T * Cin};
    a.K = P, a.R = B;
  }
  return run(a, dtype, workspace, tc_dw, (cudaStream_t)stream);
}
