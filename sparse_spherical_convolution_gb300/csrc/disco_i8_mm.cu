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

constexpr int kTile = 32, kAnyThreads = 256;

__device__ __forceinline__ float element(const Operand& o, long long i, int f16) {
  if (o.bits == 8) return (float)((const int8_t*)o.p)[i];
  return f16 ? __half2float(((const __half*)o.p)[i]) : __bfloat162float(((const __nv_bfloat16*)o.p)[i]);
}

// 32 x 32 outputs to a block, four to a thread; 32 k at a time through shared memory.
template <typename TO>
__global__ void __launch_bounds__(kAnyThreads) mm_any_kernel(const MmArgs a) {
  __shared__ float sa[kTile][kTile + 1], sb[kTile][kTile + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const long long mt = (a.M + kTile - 1) / kTile, nt = (a.N + kTile - 1) / kTile;
  const int f16 = a.f16;
  for (long long t = blockIdx.x; t < mt * nt * a.Z; t += gridDim.x) {
    const long long n0 = t % nt * kTile, m0 = t / nt % mt * kTile, z = t / (nt * mt);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int r = 0; r < a.R; ++r)
      for (long long k0 = 0; k0 < a.K; k0 += kTile) {
        // neighbouring threads read neighbouring elements: of a row, or of 32 rows' k
        auto fill = [&](const Operand& o, long long i0, long long I, float (*s)[kTile + 1]) {
          for (int u = ty; u < kTile; u += 8) {
            const int i = o.k_major ? u : tx, k = o.k_major ? tx : u;
            float v = 0.0f;
            if (i0 + i < I && k0 + k < a.K) {
              const long long zr = z * o.z + r * o.r;
              v = element(o, zr + (o.k_major ? (i0 + i) * o.ld + k0 + k : (k0 + k) * o.ld + i0 + i), f16);
              if (o.ks) v *= o.ks[r * o.ks_r + k0 + k];
            }
            s[k][i] = v;
          }
        };
        fill(a.A, m0, a.M, sa);
        fill(a.B, n0, a.N, sb);
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < kTile; ++k) {
          const float w = sb[k][tx];
#pragma unroll
          for (int u = 0; u < 4; ++u) acc[u] = fmaf(sa[k][ty + 8 * u], w, acc[u]);
        }
        __syncthreads();
      }
    const long long n = n0 + tx;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long m = m0 + ty + 8 * u;
      if (m >= a.M || n >= a.N) continue;
      float v = acc[u];
      if (a.cs) v *= a.cs[z * a.cs_z + n];
      if (a.rs) v *= a.rs[m];
      ((TO*)a.out)[(z * a.M + m) * a.N + n] = from_f32<TO>(v);
    }
  }
}

int run(const MmArgs& a, disco_dtype dtype, cudaStream_t st) {
  const long long tiles = (a.M + kTile - 1) / kTile * ((a.N + kTile - 1) / kTile) * a.Z;
  const int grid = (int)min(tiles, (long long)kSMs * 16);
#define CALL(T) mm_any_kernel<T><<<grid, kAnyThreads, 0, st>>>(a)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return check_launch("mm_any_kernel");
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
  return 16;
}

extern "C" size_t disco_matmul_i8_bwd_input_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return 16;
}

extern "C" size_t disco_matmul_i8_bwd_weight_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return 16;
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
    a.A = {q, nullptr, 0, 0, Cin, 0, 8, true};
    a.B = {W, nullptr, 0, 0, Cin, 0, 8, true};
    a.rs = scale, a.cs = wscale;
    a.M = B, a.N = Cout, a.Z = 1;
  } else {  // m = output channel, n = pixel
    a.A = {W, nullptr, 0, 0, Cin, 0, 8, true};
    a.B = {q, nullptr, Cin * P, 0, P, 0, 8, false};
    a.rs = wscale, a.cs = scale, a.cs_z = P;
    a.M = Cout, a.N = P, a.Z = B;
  }
  return run(a, dtype, (cudaStream_t)stream);
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
    a.A = {dy, nullptr, 0, 0, Cout, 0, 16, true};
    a.B = {W, wscale, 0, 0, Cin, 0, 8, false};
    a.M = B, a.N = Cin, a.Z = 1;
  } else {  // m = input channel, n = pixel
    a.A = {W, wscale, 0, 0, Cin, 0, 8, false};
    a.B = {dy, nullptr, Cout * P, 0, P, 0, 16, false};
    a.M = Cin, a.N = P, a.Z = B;
  }
  return run(a, dtype, (cudaStream_t)stream);
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
    a.A = {dy, nullptr, 0, 0, Cout, 0, 16, false};
    a.B = {q, scale, 0, 0, Cin, 0, 8, false};
    a.K = B, a.R = 1;
  } else {  // k = pixel, summed over the samples too
    a.A = {dy, nullptr, 0, Cout * P, P, 0, 16, true};
    a.B = {q, scale, 0, Cin * P, P, P, 8, true};
    a.K = P, a.R = B;
  }
  return run(a, dtype, (cudaStream_t)stream);
}
