// disco_i8_mm.cu -- products over the channels of each token with activations and
// weights in 8-bit integers, and their gradients from the 8-bit activation:
// checks, the cut into tiles and parts, operands laid out once a call, the kernel of a few
// rows, and the joining of parts.  All else goes to the tensor cores (disco_i8_tc.cuh).
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

// The largest finite scale of each block's share (Range).
__global__ void __launch_bounds__(kAnyThreads) mm_range_kernel(const float* scale, long long n, float* part) {
  __shared__ uint32_t most;
  norm::let_next_begin();
  if (threadIdx.x == 0) most = 0;
  __syncthreads();
  const uint32_t m = largest(scale, n, (long long)blockIdx.x * kAnyThreads + threadIdx.x, (long long)gridDim.x * kAnyThreads);
  if ((threadIdx.x & 31) == 0) atomicMax(&most, m);
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = __uint_as_float(most);
}

// ---- operands laid out once a call --------------------------------------------
// Bound by HBM, or by a launch: a thread writes one 16-byte word of a row, from two aligned
// words shifted together where the source's rows start anywhere.  With its
// copies and its 2-byte stores a product of 512 by 512 channels takes 184 us on 259199
// pixels and 128 on 259200.

__device__ __forceinline__ uint4 load16(const uint8_t* p, const uint8_t* end) {
  if (p + 16 <= end) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (p + i < end) w[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// `rows` rows of `len` elements of es bytes, to rows of `words` words, zeros at their
// end.  Kinds: 0 as they are; else integers to fp16 (1), or times their row's scale, rounded, to fp16 (2) or bf16 (3).
struct Layout {
  const uint8_t *src, *end;
  uint4* dst;
  const float* scale;
  long long len, words, total;
  int es, kind;
  uint32_t block0;  // the first block that works on it
};
struct Layouts {
  Layout t[3];
  int n;
  Range range;  // of the scales of kind 2
};

__global__ void __launch_bounds__(kAnyThreads) mm_layout_kernel(const Layouts a) {
  __shared__ uint32_t most;
  norm::let_next_begin();
  int k = 0;
  if (a.n > 1 && blockIdx.x >= a.t[1].block0) k = 1;
  if (a.n > 2 && blockIdx.x >= a.t[2].block0) k = 2;
  const Layout& t = a.t[k];
  const long long i = (long long)(blockIdx.x - t.block0) * kAnyThreads + threadIdx.x;
  const bool live = i < t.total;
  const long long row = t.total <= 0xffffffffLL ? (long long)((uint32_t)i / (uint32_t)t.words) : i / t.words;
  const int step = t.kind ? 8 : 16;  // source bytes of a word
  const long long at = (i - row * t.words) * step;
  const int nb = live ? (int)max(0LL, min((long long)step, t.len * t.es - at)) : 0;
  uint4 v = make_uint4(0, 0, 0, 0);
  if (nb > 0) {
    const uint8_t* p = t.src + row * t.len * t.es + at;
    const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15);
    if (DISCO_IN_BOUNDS(p - sh >= t.src && p + nb <= t.end)) {
      const uint4 lo = load16(p - sh, t.end);
      v = shifted(lo, sh + nb > 16 ? load16(p - sh + 16, t.end) : v, sh, nb);
    }
  }
  // every block waits for the range, so that this kernel's end tells the next one that it is there
  norm::wait_for_previous();
  float down = 1.0f;
  if (t.kind == 2) {
    if (threadIdx.x == 0) most = 0;
    __syncthreads();
    const uint32_t m = largest(a.range.v, a.range.n, threadIdx.x, kAnyThreads);
    if ((threadIdx.x & 31) == 0) atomicMax(&most, m);
    __syncthreads();
    down = fit_down(most);
  }
  if (!live) return;
  if (t.kind) {
    const uint32_t w[2] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u};
    const float f = t.kind > 1 ? t.scale[row] * down : 1.0f;
    auto two = [&](int e) { return pack2_16(from_byte(w[e / 4], e & 3) * f, from_byte(w[e / 4], (e & 3) + 1) * f, t.kind < 3); };
    v = make_uint4(two(0), two(2), two(4), two(6));
  }
  t.dst[i] = v;
}

// ---- a few rows ----------------------------------------------------------------
// Bound by the weight's bytes, or by the latency of one round to memory: 1 row of 512 to 2048
// channels 2.2 us (9.0 on the tensor cores), 8 rows of 2048 to 512 4.1 us (11).  A warp takes O
// output channels and all NB rows: a lane 16 input channels of each at a time, four
// products and their sum to an instruction (dp4a), exact in 32 bits.  The rows lie in shared memory
// from their first byte on, zeros behind them.
constexpr int kFewThreads = 128, kFewRows = 16;
// Rows beyond this leave too few warps to an SM: 12 rows of 8192 to 3079 channels (128 KB) took 58
// us (16 on the tensor cores), of 4096 (64 KB) 15.5 (12.3); 4 rows of 8192 (32 KB) take 8.6 (16),
// 12 of 2048 7.3 (10).  Its 2^15 products at most keep a sum in 32 bits.
constexpr size_t kFewSmem = 32 * 1024;

// Word i (16 bytes) of a row of C bytes anywhere in a tensor that ends at `end`.
template <bool ALN>
__device__ __forceinline__ uint4 row_word(const uint8_t* row, int i, int C, const uint8_t* end) {
  if (ALN) return __ldg(reinterpret_cast<const uint4*>(row) + i);
  const uint8_t* p = row + 16 * i;
  const int sh = (int)(reinterpret_cast<uintptr_t>(p) & 15), nb = min(16, C - 16 * i);
  if (nb <= 0) return make_uint4(0, 0, 0, 0);
  const uint4 lo = load16(p - sh, end);
  return shifted(lo, sh + nb > 16 ? load16(p - sh + 16, end) : make_uint4(0, 0, 0, 0), sh, nb);
}

struct FewArgs {
  const uint8_t *q, *W;
  const float *scale, *wscale;
  void* y;
  int B, Cin, Cout, type;
};

template <int NB, int O, bool ALN>
__global__ void __launch_bounds__(kFewThreads) mm_few_kernel(const FewArgs a) {
  extern __shared__ __align__(16) uint4 rows[];  // [NB][words]
  const int lane = threadIdx.x & 31, words = (a.Cin + 15) / 16;
  const int o0 = (blockIdx.x * (kFewThreads / 32) + threadIdx.x / 32) * O;
  const uint8_t *qend = a.q + (long long)a.B * a.Cin, *wend = a.W + (long long)a.Cout * a.Cin;
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
  return P == 1 && B <= kFewRows && (size_t)NB * ((Cin + 15) / 16) * 16 <= kFewSmem;
}

// As many scales each block of the kernels that need the largest one reads for itself; of more, mm_range_kernel's
// parts.  dx of 512 rows 1024 -> 4096 takes 19.9 us with the parts, 21.4 without; 4 x 64 -> 48 on 33x65 6.4
// without, 7.6 with them.  (5.7 and 17.8 if the scales stayed as they are.)
constexpr long long kRangeDirect = 1024;

// The cut of a product by its sizes alone (the workspace's bytes follow from it).
// Tiles of 256 n; where they do not fill the SMs, the reduction is split into parts of 8 steps
// at least (2 where the sums are few), and where that leaves half of the SMs idle, tiles get narrower.
// No part has more than kPartSteps; where that decides, parts are added until they fill the SMs evenly.
struct Cut {
  int NB;
  long long nsplit, mt, nt, nkp, steps;
  Cut(long long M, long long N, long long K, int Z, int R) {
    mt = (M + 127) / 128;
    nkp = (K + 63) / 64;
    steps = nkp * R;
    NB = N >= 256 ? 256 : (int)((N + 15) / 16 * 16);
    for (;;) {
      nt = (N + NB - 1) / NB;
      const long long tiles = mt * nt * Z;
      nsplit = max(1LL, min(steps / (M * N * Z <= 1 << 16 ? 2 : 8), kSMs / tiles));
      if (tiles * nsplit >= kSMs / 2 || NB <= 64) break;
      NB = NB > 128 ? 128 : 64;
    }
    const long long least = (steps + kPartSteps - 1) / kPartSteps, tiles = mt * nt * Z;
    if (nsplit < least) nsplit = max(least, (least * tiles + kSMs - 1) / kSMs * kSMs / tiles);
  }
};

// A product ready to launch: its arguments, the operands that are laid out first, and the bytes of
// the workspace it takes.  Made from the sizes alone where `ws` is null.
struct Product {
  MmArgs m = {};
  Cut cut;
  Layouts lay = {};
  char* ws;
  size_t bytes = 0;
  uint32_t blocks = 0;
  const float* scales = nullptr;
  long long nscales = 0;

  Product(void* workspace, long long M, long long N, long long K, int Z, int R, bool transposed) : cut(M, N, K, Z, R), ws((char*)workspace) {
    m.M = M, m.N = N, m.K = K, m.Z = Z, m.R = R, m.transposed = transposed;
  }
  void* take(size_t n) {
    void* p = ws ? ws + bytes : nullptr;
    bytes += (n + 255) / 256 * 256;
    return p;
  }
  void* add(const void* src, const float* scale, long long rows, long long len, long long words, int es, int kind) {
    Layout& t = lay.t[lay.n++];
    t.src = (const uint8_t*)src, t.end = t.src + rows * len * es;
    t.scale = scale, t.len = len, t.words = words, t.total = rows * words, t.es = es, t.kind = kind;
    t.block0 = blocks;
    blocks += (uint32_t)((t.total + kAnyThreads - 1) / kAnyThreads);
    t.dst = (uint4*)take((size_t)t.total * 16);
    return t.dst;
  }
  // [rows][ld] as it is where rows start on 16 bytes, else a copy that does
  Operand rows(Operand o, long long rows) {
    const int es = o.bits / 8;
    if (o.ld * es % 16 == 0) return o;
    const long long words = (o.ld * es + 15) / 16, pitch = words * 16 / es;
    o.p = add(o.p, nullptr, rows, o.ld, words, es, 0);
    o.z = o.z / o.ld * pitch, o.r = o.r / o.ld * pitch, o.ld = pitch;
    return o;
  }
  // integers [rows][C] in 16 bits; scaled: times their row's scale
  Operand halves(const void* q, bool scaled, const float* scale, long long rows, long long C, bool f16, bool k_major) {
    const long long words = (C + 7) / 8;
    return {add(q, scale, rows, C, words, 1, !scaled ? 1 : f16 ? 2 : 3), nullptr, 0, 0, words * 8, 0, 16, k_major};
  }
  // fp16 gradients: the range of n scales (its words are taken for every type: one size for all)
  void ranged(const float* scale, long long n) {
    float* p = (float*)take(kSMs * 4);
    if (!m.f16) return;
    if (n <= kRangeDirect) {
      m.range = {scale, (int)n};
      return;
    }
    scales = scale, nscales = n;
    m.range = {p, kSMs};
  }
  float* parts() { return cut.nsplit > 1 ? (float*)take((size_t)cut.nsplit * m.Z * m.M * m.N * 4) : nullptr; }

  int run(float* part, disco_dtype dtype, int (*tc)(const TcArgs&, cudaStream_t), cudaStream_t st) const {
    if (cut.mt * cut.nt * m.Z * cut.nsplit >= 1LL << 31) return fail(DISCO_ERR_UNSUPPORTED, "more than 2^31 tiles of 128 by %d", cut.NB);
    if (scales) {
      mm_range_kernel<<<kSMs, kAnyThreads, 0, st>>>(scales, nscales, const_cast<float*>(m.range.v));
      if (int rc = check_launch("mm_range_kernel")) return rc;
    }
    if (lay.n) {
      if (int rc = norm::launch(mm_layout_kernel, (int)blocks, kAnyThreads, 1, scales != nullptr, 0, 0, st, "mm_layout_kernel", lay)) return rc;
    }
    TcArgs a = {};
    a.m = m;
    a.NB = cut.NB, a.nsplit = (int)cut.nsplit, a.mt = (uint32_t)cut.mt, a.nt = (uint32_t)cut.nt, a.nkp = cut.nkp, a.steps = cut.steps;
    a.part = cut.nsplit > 1 ? part : nullptr;
    a.out_type = dtype;
    a.after = lay.n > 0 || scales;
    a.vec = (m.transposed ? m.M : m.N) * (a.part ? 4 : elem_bytes(dtype)) % 16 == 0;
    a.tiles = (uint32_t)(cut.mt * cut.nt * m.Z * cut.nsplit);
    int rc = tc(a, st);
    if (rc || !a.part) return rc;
    const long long n = m.Z * m.M * m.N;
    const int grid = (int)min((n + kAnyThreads - 1) / kAnyThreads, (long long)kSMs * 8);
#define CALL(T) rc = norm::launch(mm_join_kernel<T>, grid, kAnyThreads, 1, true, 0, 0, st, "mm_join_kernel", m, (const float*)part, (int)cut.nsplit, n)
    DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
    return rc;
  }
};

// Of the product of rows, the smaller operand is converted once a call, the other one in the main loop.
Product product(const void* q, const float* scale, const void* W, const float* wscale, void* y, int32_t B, int32_t Cin, int32_t Cout,
                int64_t P, void* ws, float** part) {
  const bool swap = P == 1 && B < Cout;
  Product p = swap ? Product(ws, Cout, B, Cin, 1, 1, true) : P == 1 ? Product(ws, B, Cout, Cin, 1, 1, false) : Product(ws, P, Cout, Cin, B, 1, true);
  p.m.out = y;
  p.m.rs = swap ? wscale : scale, p.m.cs = swap ? scale : wscale;
  if (swap) {  // m = output channel, n = row
    p.m.A = p.rows({W, nullptr, 0, 0, Cin, 0, 8, true}, Cout);
    p.m.B = p.halves(q, false, nullptr, B, Cin, true, true);
  } else {
    p.m.B = p.halves(W, false, nullptr, Cout, Cin, true, true);
    if (P == 1) {  // m = row
      p.m.A = p.rows({q, nullptr, 0, 0, Cin, 0, 8, true}, B);
    } else {  // m = pixel
      p.m.A = p.rows({q, nullptr, Cin * P, 0, P, 0, 8, false}, (long long)B * Cin);
      p.m.rs_z = P;
    }
  }
  *part = p.parts();
  return p;
}
Product product_dx(const void* dy, const void* W, const float* wscale, void* dx, int32_t B, int32_t Cin, int32_t Cout, int64_t P, bool f16,
                   void* ws, float** part) {
  Product p = P == 1 ? Product(ws, B, Cin, Cout, 1, 1, false) : Product(ws, P, Cin, Cout, B, 1, true);
  p.m.out = dx;
  p.m.f16 = f16;
  p.ranged(wscale, Cout);
  p.lay.range = p.m.range;
  p.m.B = p.halves(W, true, wscale, Cout, Cin, f16, false);
  if (P == 1) p.m.A = p.rows({dy, nullptr, 0, 0, Cout, 0, 16, true}, B);  // m = row
  else p.m.A = p.rows({dy, nullptr, Cout * P, 0, P, 0, 16, false}, (long long)B * Cout);  // m = pixel
  *part = p.parts();
  return p;
}
Product product_dw(const void* dy, const void* q, const float* scale, void* dW, int32_t B, int32_t Cin, int32_t Cout, int64_t P, bool f16,
                   void* ws, float** part) {
  Product p = P == 1 ? Product(ws, Cin, Cout, B, 1, 1, true) : Product(ws, Cin, Cout, P, 1, B, true);  // m = input channel
  p.m.out = dW;
  p.m.f16 = f16;
  p.ranged(scale, (long long)B * P);
  if (P == 1) {  // k = row
    p.m.A = p.rows({q, scale, 0, 0, Cin, 0, 8, false}, B);
    p.m.B = p.rows({dy, nullptr, 0, 0, Cout, 0, 16, false}, B);
  } else {  // k = pixel, summed over the samples too
    p.m.A = p.rows({q, scale, 0, Cin * P, P, P, 8, true}, (long long)B * Cin);
    p.m.B = p.rows({dy, nullptr, 0, Cout * P, P, 0, 16, true}, (long long)B * Cout);
    if (P % 16) {  // rows of scales that go on in zeros
      const long long words = (P + 15) / 16 * 4;
      p.m.A.ks = (const float*)p.add(scale, nullptr, B, P, words, 4, 0);
      p.m.A.ks_r = words * 4;
    }
  }
  *part = p.parts();
  return p;
}

// Sizes of a product; 16-bit types only for the gradients.
int check_mm(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype, bool grad) {
  int rc;
  if ((rc = check_shape(B, Cin, P, dtype)) || (rc = check_shape(B, Cout, P, dtype))) return rc;
  if (grad && dtype == DISCO_F32) return fail(DISCO_ERR_UNSUPPORTED, "gradients take bf16 or fp16");
  if ((double)Cin * Cout > 1e12) return fail(DISCO_ERR_UNSUPPORTED, "more than 1e12 weights");
  // the copy engine's coordinates are 32-bit, its strides below 2^40 bytes
  if (P >= 1LL << 31 || (double)max(Cin, Cout) * (double)P * 2 >= 1099511627776.0)
    return fail(DISCO_ERR_UNSUPPORTED, "2^31 pixels or more, or 2^40 bytes of a sample");
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
  float* part;
  return product(nullptr, nullptr, nullptr, nullptr, nullptr, B, Cin, Cout, P, nullptr, &part).bytes;
}

extern "C" size_t disco_matmul_i8_bwd_input_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  float* part;
  return product_dx(nullptr, nullptr, nullptr, nullptr, B, Cin, Cout, P, false, nullptr, &part).bytes;
}

extern "C" size_t disco_matmul_i8_bwd_weight_workspace_bytes(int32_t B, int32_t Cin, int32_t Cout, int64_t P, disco_dtype dtype) {
  if (check_mm(B, Cin, Cout, P, dtype, true)) return 0;
  float* part;
  return max((size_t)16, product_dw(nullptr, nullptr, nullptr, nullptr, B, Cin, Cout, P, false, nullptr, &part).bytes);
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
    const FewArgs a{(const uint8_t*)q, (const uint8_t*)W, scale, wscale, y, B, Cin, Cout, dtype};
    return B == 1 ? few<1>(a, st) : B <= 4 ? few<4>(a, st) : few<16>(a, st);
  }
  float* part;
  const Product p = product(q, scale, W, wscale, y, B, Cin, Cout, P, workspace, &part);
  return p.run(part, dtype, tc_fwd, st);
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
  float* part;
  const Product p = product_dx(dy, W, wscale, dx, B, Cin, Cout, P, dtype == DISCO_F16, workspace, &part);
  return p.run(part, dtype, tc_dx, (cudaStream_t)stream);
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
  float* part;
  const Product p = product_dw(dy, q, scale, dW, B, Cin, Cout, P, dtype == DISCO_F16, workspace, &part);
  return p.run(part, dtype, tc_dw, (cudaStream_t)stream);
}
