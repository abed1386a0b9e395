// disco_i8_mm.cu -- products over the channels of each token with activations and
// weights in 8-bit integers, and their gradients from the 8-bit activation:
// checks, the choice of a kernel, and the general one.
//
//   y[b,o,p]  = scale[b,p] wscale[o] sum_c W[o,c] q[b,c,p]      (disco_matmul_i8)
//   dx[b,c,p] = sum_o wscale[o] W[o,c] dy[b,o,p]                (disco_matmul_i8_bwd_input)
//   dW[o,c]   = sum_{b,p} dy[b,o,p] scale[b,p] q[b,c,p]         (disco_matmul_i8_bwd_weight)
//
// Each is a product sum_k A(m, k) B(n, k) with scales on m, n or A's k, A the
// activation (m = token; the channel of its weight's gradient).

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
    if (a.cs) {
      const long long cols = a.transposed ? a.M : a.N, rows = a.transposed ? a.N : a.M;
      const long long r = i / cols, c = i - r * cols, z = r / rows, rr = r - z * rows;
      v *= a.cs[a.transposed ? rr : c];
      v *= a.rs[z * a.rs_z + (a.transposed ? c : rr)];
    }
    ((TO*)a.out)[i] = from_f32<TO>(v);
  }
}

// A weight [Cout][Cin] as the 16-bit operand: the integers in fp16, or times their
// channel's scale rounded to the type; rows padded to `ld` elements with zeros.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) mm_weight_kernel(const int8_t* W, const float* wscale, T* w16, int Cin, int ld, long long n) {
  const long long i = ((long long)blockIdx.x * kAnyThreads + threadIdx.x) * 8;
  if (i >= n) return;
  const long long o = i / ld;
  const int c = (int)(i - o * ld);
  const float f = wscale ? wscale[o] : 1.0f;
  T v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = from_f32<T>(c + e < Cin ? (float)W[o * Cin + c + e] * f : 0.0f);
  *reinterpret_cast<uint4*>(w16 + i) = *reinterpret_cast<const uint4*>(v);
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
    NB = N >= 256 ? 256 : (int)((N + 15) / 16 * 16);
    for (;;) {
      nt = (N + NB - 1) / NB;
      const long long tiles = mt * nt * Z;
      nsplit = (int)max(1LL, min(steps / 8, kSMs / tiles));
      if (tiles * nsplit >= kSMs / 2 || NB <= 64) break;
      NB = NB > 128 ? 128 : 64;
    }
  }
  size_t part_bytes(long long M, long long N, int Z) const { return nsplit > 1 ? (size_t)nsplit * Z * M * N * 4 : 0; }
};

// What a call needs of the workspace: the 16-bit weight, then the parts' sums.
size_t weight_bytes(int32_t Cin, int32_t Cout) { return ((size_t)Cout * (((size_t)Cin + 7) / 8 * 8) * 2 + 255) / 256 * 256; }

Cut cut_fwd(int32_t B, int32_t Cin, int32_t Cout, int64_t P) { return P == 1 ? Cut(B, Cout, Cin, 1, 1) : Cut(P, Cout, Cin, B, 1); }
Cut cut_dx(int32_t B, int32_t Cin, int32_t Cout, int64_t P) { return P == 1 ? Cut(B, Cin, Cout, 1, 1) : Cut(P, Cin, Cout, B, 1); }
Cut cut_dw(int32_t B, int32_t Cin, int32_t Cout, int64_t P) { return P == 1 ? Cut(Cin, Cout, B, 1, 1) : Cut(Cin, Cout, P, 1, B); }

bool rows_aligned(const Operand& o) {
  const int es = o.bits / 8;
  return o.ld * es % 16 == 0 && o.z * es % 16 == 0 && o.r * es % 16 == 0;
}

int run(const MmArgs& m, const Cut& c, disco_dtype dtype, void* part, int (*tc)(const TcArgs&, cudaStream_t), cudaStream_t st) {
  if (c.mt * c.nt * m.Z * c.nsplit >= 1LL << 31) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^31 tiles of 128 by %d", c.NB);
  TcArgs a = {};
  a.m = m;
  a.enda = (const uint8_t*)m.A.p + m.A.n * (m.A.bits / 8);
  a.endb = (const uint8_t*)m.B.p + m.B.n * (m.B.bits / 8);
  a.NB = c.NB, a.nsplit = c.nsplit, a.mt = (uint32_t)c.mt, a.nt = (uint32_t)c.nt, a.nkp = c.nkp, a.steps = c.steps;
  a.part = c.nsplit > 1 ? (float*)part : nullptr;
  a.out_type = dtype;
  a.vec = (m.transposed ? m.M : m.N) * (a.part ? 4 : elem_bytes(dtype)) % 16 == 0;
  a.tiles = (uint32_t)(c.mt * c.nt * m.Z * c.nsplit);
  // the copy engine's coordinates are 32-bit, its strides below 2^40 bytes
  const bool small = max(max(m.M, m.N), m.K) < 1LL << 31 && max(m.A.n, m.B.n) < 1LL << 38;
  a.ala = small && rows_aligned(m.A), a.alb = small && rows_aligned(m.B);
  int rc = tc(a, st);
  if (rc || !a.part) return rc;
  const long long n = m.Z * m.M * m.N;
  const int grid = (int)min((n + kAnyThreads - 1) / kAnyThreads, (long long)kSMs * 8);
#define CALL(T) mm_join_kernel<T><<<grid, kAnyThreads, 0, st>>>(m, a.part, c.nsplit, n)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("mm_join_kernel");
}

int weight_16(const void* W, const float* wscale, void* w16, int32_t Cin, int32_t Cout, bool f16, cudaStream_t st) {
  const int ld = (int)(((long long)Cin + 7) / 8 * 8);
  const long long n = (long long)Cout * ld, grid = (n / 8 + kAnyThreads - 1) / kAnyThreads;
  if (f16) mm_weight_kernel<<<(unsigned)grid, kAnyThreads, 0, st>>>((const int8_t*)W, wscale, (__half*)w16, Cin, ld, n);
  else mm_weight_kernel<<<(unsigned)grid, kAnyThreads, 0, st>>>((const int8_t*)W, wscale, (__nv_bfloat16*)w16, Cin, ld, n);
  return check_launch("mm_weight_kernel");
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
  return weight_bytes(Cin, Cout) + cut_fwd(B, Cin, Cout, P).part_bytes((long long)B * P, Cout, 1);
}

extern "C" size_t disco_matmul_i8_bwd_input_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return weight_bytes(Cin, Cout) + cut_dx(B, Cin, Cout, P).part_bytes((long long)B * P, Cin, 1);
}

extern "C" size_t disco_matmul_i8_bwd_weight_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return max((size_t)16, cut_dw(B, Cin, Cout, P).part_bytes(Cin, Cout, 1));
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
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = weight_16(W, nullptr, workspace, Cin, Cout, true, st))) return rc;
  const long long ld = ((long long)Cin + 7) / 8 * 8;
  MmArgs a = {};
  a.out = y;
  a.rs = scale, a.cs = wscale;
  a.N = Cout, a.K = Cin, a.R = 1;
  a.B = {workspace, nullptr, 0, 0, ld, 0, 16, true, Cout * ld};
  if (P == 1) {  // m = row
    a.A = {q, nullptr, 0, 0, Cin, 0, 8, true, (long long)(T * Cin)};
    a.M = B, a.Z = 1;
  } else {  // m = pixel
    a.A = {q, nullptr, Cin * P, 0, P, 0, 8, false, (long long)(T * Cin)};
    a.M = P, a.Z = B, a.rs_z = P, a.transposed = true;
  }
  return run(a, cut_fwd(B, Cin, Cout, P), dtype, (char*)workspace + weight_bytes(Cin, Cout), tc_fwd, st);
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
  const cudaStream_t st = (cudaStream_t)stream;
  if ((rc = weight_16(W, wscale, workspace, Cin, Cout, dtype == DISCO_F16, st))) return rc;
  const long long ld = ((long long)Cin + 7) / 8 * 8;
  MmArgs a = {};
  a.out = dx;
  a.f16 = dtype == DISCO_F16;
  a.N = Cin, a.K = Cout, a.R = 1;
  a.B = {workspace, nullptr, 0, 0, ld, 0, 16, false, Cout * ld};
  if (P == 1) {  // m = row
    a.A = {dy, nullptr, 0, 0, Cout, 0, 16, true, (long long)(T * Cout)};
    a.M = B, a.Z = 1;
  } else {  // m = pixel
    a.A = {dy, nullptr, Cout * P, 0, P, 0, 16, false, (long long)(T * Cout)};
    a.M = P, a.Z = B, a.transposed = true;
  }
  return run(a, cut_dx(B, Cin, Cout, P), dtype, (char*)workspace + weight_bytes(Cin, Cout), tc_dx, st);
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
  a.M = Cin, a.N = Cout, a.Z = 1, a.transposed = true;  // m = input channel
  if (P == 1) {  // k = row
    a.A = {q, scale, 0, 0, Cin, 0, 8, false, (long long)(T * Cin)};
    a.B = {dy, nullptr, 0, 0, Cout, 0, 16, false, (long long)(T * Cout)};
    a.K = B, a.R = 1;
  } else {  // k = pixel, summed over the samples too
    a.A = {q, scale, 0, Cin * P, P, P, 8, true, (long long)(T * Cin)};
    a.B = {dy, nullptr, 0, Cout * P, P, 0, 16, true, (long long)(T * Cout)};
    a.K = P, a.R = B;
  }
  return run(a, cut_dw(B, Cin, Cout, P), dtype, workspace, tc_dw, (cudaStream_t)stream);
}
