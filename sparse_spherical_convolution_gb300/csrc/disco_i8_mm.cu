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
#include "disco_umma.cuh"

namespace disco {

DISCO_BOUNDS_READER(i8_mm_bounds)

namespace {

using namespace i8;

constexpr int kAnyThreads = 256;

// The parts' sums in their order, scaled and rounded.
template <typename TO>
__global__ void __launch_bounds__(kAnyThreads) mm_join_kernel(const MmArgs a, const float* part, int nsplit, long long n) {
  norm::wait_for_previous();
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

// Integers [rows][C] as the 16-bit operand: in fp16, or times their row's scale rounded
// to the type; rows padded to `ld` elements with zeros.
template <typename T>
__global__ void __launch_bounds__(kAnyThreads) mm_operand_kernel(const int8_t* q, const float* scale, T* w16, int C, int ld, long long n) {
  const long long i = ((long long)blockIdx.x * kAnyThreads + threadIdx.x) * 8;
  norm::let_next_begin();
  if (i >= n) return;
  const long long o = n <= 0xffffffffLL ? (long long)((uint32_t)i / (uint32_t)ld) : i / ld;
  const int c = (int)(i - o * ld);
  const float f = scale ? scale[o] : 1.0f;
  uint32_t w[2];
  if (C % 8 == 0) {
    const uint2 u = *reinterpret_cast<const uint2*>(q + i);
    w[0] = u.x, w[1] = u.y;
  } else {
    w[0] = w[1] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < C) w[e / 4] |= (uint32_t)(uint8_t)q[o * C + c + e] << (8 * (e & 3));
  }
  T v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = from_f32<T>(from_byte(w[e / 4] ^ 0x80808080u, e & 3) * f);
  *reinterpret_cast<uint4*>(w16 + i) = *reinterpret_cast<const uint4*>(v);
}

// ---- a few rows ----------------------------------------------------------------
// Bound by the weight's bytes, or by the latency of one round to memory.  A warp takes O
// output channels and all NB rows: a lane 16 input channels of each at a time, four
// products and their sum to an instruction (dp4a), exact in 32 bits.  The rows lie in shared memory
// from their first byte on, zeros behind them.
constexpr int kFewThreads = 128, kFewRows = 16;
constexpr size_t kFewSmem = 128 * 1024;

__device__ __forceinline__ uint4 load16(const int8_t* p, const int8_t* end) {
  if (p + 16 <= end) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (p + i < end) w[i >> 2] |= (uint32_t)(uint8_t)p[i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Word i (16 bytes) of a row of C bytes anywhere in a tensor that ends at `end`.
template <bool ALN>
__device__ __forceinline__ uint4 row_word(const int8_t* row, int i, int C, const int8_t* end) {
  if (ALN) return __ldg(reinterpret_cast<const uint4*>(row) + i);
  const int8_t* p = row + 16 * i;
  const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15), nb = min(16, C - 16 * i);
  if (nb <= 0) return make_uint4(0, 0, 0, 0);
  const uint4 lo = load16(p - sh, end);
  return shifted(lo, sh + nb > 16 ? load16(p - sh + 16, end) : make_uint4(0, 0, 0, 0), sh, nb);
}

struct FewArgs {
  const int8_t *q, *W;
  const float *scale, *wscale;
  void* y;
  int B, Cin, Cout, type;
};

template <int NB, int O, bool ALN>
__global__ void __launch_bounds__(kFewThreads) mm_few_kernel(const FewArgs a) {
  extern __shared__ __align__(16) uint4 rows[];  // [NB][words]
  const int lane = threadIdx.x & 31, words = (a.Cin + 15) / 16;
  const int o0 = (blockIdx.x * (kFewThreads / 32) + threadIdx.x / 32) * O;
  const int8_t *qend = a.q + (long long)a.B * a.Cin, *wend = a.W + (long long)a.Cout * a.Cin;
  uint4 w[O];
  auto fetch = [&](int i) {
#pragma unroll
    for (int k = 0; k < O; ++k)
      w[k] = o0 + k < a.Cout && i < words ? row_word<ALN>(a.W + (long long)(o0 + k) * a.Cin, i, a.Cin, wend) : make_uint4(0, 0, 0, 0);
  };
  fetch(lane);
  for (int i = threadIdx.x; i < NB * words; i += kFewThreads) {
    const int b = i / words;
    rows[i] = b < a.B ? row_word<ALN>(a.q + (long long)b * a.Cin, i - b * words, a.Cin, qend) : make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  int acc[O][NB] = {};
  for (int i = lane; i < words; i += 32) {
    uint4 v[O];
#pragma unroll
    for (int k = 0; k < O; ++k) v[k] = w[k];
    fetch(i + 32);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 x = rows[b * words + i];
#pragma unroll
      for (int k = 0; k < O; ++k)
        acc[k][b] = __dp4a((int)v[k].w, (int)x.w, __dp4a((int)v[k].z, (int)x.z, __dp4a((int)v[k].y, (int)x.y, __dp4a((int)v[k].x, (int)x.x, acc[k][b]))));
    }
  }
  int mine[(O * NB + 31) / 32] = {};  // output k NB + b goes to lane (k NB + b) % 32
#pragma unroll
  for (int k = 0; k < O; ++k)
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int s = __reduce_add_sync(0xffffffffu, acc[k][b]), at = k * NB + b;
      if (lane == at % 32) mine[at / 32] = s;
    }
#pragma unroll
  for (int m = 0; m < (O * NB + 31) / 32; ++m) {
    const int at = lane + 32 * m, b = at % NB, o = o0 + at / NB;
    if (at < O * NB && b < a.B && o < a.Cout) {
      const float v = (float)mine[m] * a.wscale[o] * a.scale[b];
      const long long i = (long long)b * a.Cout + o;
      if (a.type == DISCO_F32) ((float*)a.y)[i] = v;
      else ((uint16_t*)a.y)[i] = round_16(v, a.type == DISCO_F16);
    }
  }
}

template <int NB, int O>
int few(const FewArgs& a, cudaStream_t st) {
  const int grid = (a.Cout + kFewThreads / 32 * O - 1) / (kFewThreads / 32 * O);
  const size_t smem = (size_t)NB * ((a.Cin + 15) / 16) * 16;
  if (a.Cin % 16 == 0) return norm::launch(mm_few_kernel<NB, O, true>, grid, kFewThreads, 1, false, smem, kFewSmem, st, "mm_few_kernel", a);
  return norm::launch(mm_few_kernel<NB, O, false>, grid, kFewThreads, 1, false, smem, kFewSmem, st, "mm_few_kernel", a);
}
template <int NB>
int few(const FewArgs& a, cudaStream_t st) {
  // several channels to a warp share its reads of the rows, while every SM keeps some warps
  return a.Cout >= 8 * 4 * kSMs ? few<NB, 4>(a, st) : few<NB, 1>(a, st);
}
bool takes_few(int32_t B, int32_t Cin, int64_t P) {
  const int NB = B == 1 ? 1 : B <= 4 ? 4 : 16;
  // 32 bits hold the sum of 2^16 products
  return P == 1 && B <= kFewRows && Cin <= 1 << 16 && (size_t)NB * ((Cin + 15) / 16) * 16 <= kFewSmem;
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

// What a call needs of the workspace: the 16-bit operand, then the parts' sums.
size_t operand_bytes(long long rows, int32_t C) { return ((size_t)rows * (((size_t)C + 7) / 8 * 8) * 2 + 255) / 256 * 256; }
// Of the product of rows, the smaller operand is converted once a call, the other one in the main loop.
bool rows_are_b(int32_t B, int32_t Cout, int64_t P) { return P == 1 && B < Cout; }

Cut cut_fwd(int32_t B, int32_t Cin, int32_t Cout, int64_t P) {
  return rows_are_b(B, Cout, P) ? Cut(Cout, B, Cin, 1, 1) : P == 1 ? Cut(B, Cout, Cin, 1, 1) : Cut(P, Cout, Cin, B, 1);
}
Cut cut_dx(int32_t B, int32_t Cin, int32_t Cout, int64_t P) { return P == 1 ? Cut(B, Cin, Cout, 1, 1) : Cut(P, Cin, Cout, B, 1); }
Cut cut_dw(int32_t B, int32_t Cin, int32_t Cout, int64_t P) { return P == 1 ? Cut(Cin, Cout, B, 1, 1) : Cut(Cin, Cout, P, 1, B); }

bool rows_aligned(const Operand& o) {
  const int es = o.bits / 8;
  return o.ld * es % 16 == 0 && o.z * es % 16 == 0 && o.r * es % 16 == 0;
}

// after: an operand was converted just before
int run(const MmArgs& m, const Cut& c, disco_dtype dtype, void* part, bool after, int (*tc)(const TcArgs&, cudaStream_t), cudaStream_t st) {
  if (c.mt * c.nt * m.Z * c.nsplit >= 1LL << 31) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^31 tiles of 128 by %d", c.NB);
  TcArgs a = {};
  a.m = m;
  a.enda = (const uint8_t*)m.A.p + m.A.n * (m.A.bits / 8);
  a.endb = (const uint8_t*)m.B.p + m.B.n * (m.B.bits / 8);
  a.NB = c.NB, a.nsplit = c.nsplit, a.mt = (uint32_t)c.mt, a.nt = (uint32_t)c.nt, a.nkp = c.nkp, a.steps = c.steps;
  a.part = c.nsplit > 1 ? (float*)part : nullptr;
  a.out_type = dtype;
  a.after = after;
  a.vec = (m.transposed ? m.M : m.N) * (a.part ? 4 : elem_bytes(dtype)) % 16 == 0;
  a.tiles = (uint32_t)(c.mt * c.nt * m.Z * c.nsplit);
  // the copy engine's coordinates are 32-bit, its strides below 2^40 bytes
  const bool small = max(max(m.M, m.N), m.K) < 1LL << 31 && max(m.A.n, m.B.n) < 1LL << 38;
  a.ala = small && rows_aligned(m.A), a.alb = small && rows_aligned(m.B);
  int rc = tc(a, st);
  if (rc || !a.part) return rc;
  const long long n = m.Z * m.M * m.N;
  const int grid = (int)min((n + kAnyThreads - 1) / kAnyThreads, (long long)kSMs * 8);
#define CALL(T) rc = norm::launch(mm_join_kernel<T>, grid, kAnyThreads, 1, true, 0, 0, st, "mm_join_kernel", m, (const float*)a.part, c.nsplit, n)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}

int operand_16(const void* q, const float* scale, void* w16, int32_t C, int32_t rows, bool f16, cudaStream_t st) {
  const int ld = (int)(((long long)C + 7) / 8 * 8);
  const long long n = (long long)rows * ld, grid = (n / 8 + kAnyThreads - 1) / kAnyThreads;
  if (f16) mm_operand_kernel<<<(unsigned)grid, kAnyThreads, 0, st>>>((const int8_t*)q, scale, (__half*)w16, C, ld, n);
  else mm_operand_kernel<<<(unsigned)grid, kAnyThreads, 0, st>>>((const int8_t*)q, scale, (__nv_bfloat16*)w16, C, ld, n);
  return check_launch("mm_operand_kernel");
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
  if (takes_few(B, Cin, P)) return 16;
  return operand_bytes(rows_are_b(B, Cout, P) ? B : Cout, Cin) + cut_fwd(B, Cin, Cout, P).part_bytes((long long)B * P, Cout, 1);
}

extern "C" size_t disco_matmul_i8_bwd_input_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  return operand_bytes(Cout, Cin) + cut_dx(B, Cin, Cout, P).part_bytes((long long)B * P, Cin, 1);
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
  if (takes_few(B, Cin, P)) {
    const FewArgs a{(const int8_t*)q, (const int8_t*)W, scale, wscale, y, B, Cin, Cout, dtype};
    return B == 1 ? few<1>(a, st) : B <= 4 ? few<4>(a, st) : few<16>(a, st);
  }
  const bool swap = rows_are_b(B, Cout, P);
  const long long ld = ((long long)Cin + 7) / 8 * 8, rows16 = swap ? B : Cout;
  if ((rc = operand_16(swap ? q : W, nullptr, workspace, Cin, (int32_t)rows16, true, st))) return rc;
  MmArgs a = {};
  a.out = y;
  a.K = Cin, a.R = 1, a.Z = 1;
  a.B = {workspace, nullptr, 0, 0, ld, 0, 16, true, rows16 * ld};
  if (swap) {  // m = output channel, n = row
    a.A = {W, nullptr, 0, 0, Cin, 0, 8, true, (long long)w};
    a.rs = wscale, a.cs = scale;
    a.M = Cout, a.N = B, a.transposed = true;
  } else {  // n = output channel
    a.rs = scale, a.cs = wscale;
    a.N = Cout;
    if (P == 1) {  // m = row
      a.A = {q, nullptr, 0, 0, Cin, 0, 8, true, (long long)(T * Cin)};
      a.M = B;
    } else {  // m = pixel
      a.A = {q, nullptr, Cin * P, 0, P, 0, 8, false, (long long)(T * Cin)};
      a.M = P, a.Z = B, a.rs_z = P, a.transposed = true;
    }
  }
  return run(a, cut_fwd(B, Cin, Cout, P), dtype, (char*)workspace + operand_bytes(rows16, Cin), true, tc_fwd, st);
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
  if ((rc = operand_16(W, wscale, workspace, Cin, Cout, dtype == DISCO_F16, st))) return rc;
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
  return run(a, cut_dx(B, Cin, Cout, P), dtype, (char*)workspace + operand_bytes(Cout, Cin), true, tc_dx, st);
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
  return run(a, cut_dw(B, Cin, Cout, P), dtype, workspace, false, tc_dw, (cudaStream_t)stream);
}
