// disco_dequant.cu -- the activation that the channel norm's 8-bit copy stands
// for (disco_dequant_e4m3): x = q scale.
//
// Bound by HBM: 1 byte read and 2 or 4 written to an element, and the scales.
// A thread takes V neighbouring pixels of kRun channels of one group, so the
// scales are read once for the run; its kRun loads of q are in flight together.
// Where V does not divide P the words are not pixels (rows off alignment,
// disco_norm.cuh) and a run's channels lie `apart` apart: one skew, one V scales.
//
// Measured (GB300): [2,128,361x720] to bf16 34 us, 6.1 TB/s; [2,128,361x719] (odd
// rows) 61 us, 3.4 TB/s; rows: [16384,2048], groups of 128, 24.6 us, 4.1 TB/s;
// [2355,9477] to fp16, groups of 16, 28.9 us, 2.5 TB/s (scales are looked up element
// by element).

#include "disco_norm.cuh"

namespace disco {

DISCO_BOUNDS_READER(dequant_bounds)

namespace {

using namespace norm;

constexpr int kThreads = 256;
constexpr int kRun = 8;

struct DequantArgs {
  const uint8_t* q;
  const float* scale;
  void* x;
  int G, NG, B, C;
  long long P, n;
};

// Blocks of LX lanes x J runs.  Runs of a sample: per_group of each group.
struct Cut {
  int LX, J, TP, per_group, apart;
  long long runs, run_blocks, px_tiles, blocks;  // of a sample; of the call
};

// SHIFT: V does not divide P (rows off alignment, disco_norm.cuh).
template <typename T, bool SHIFT>
__global__ void __launch_bounds__(kThreads) dequant_kernel(const DequantArgs a, const Cut g) {
  constexpr int V = 16 / (int)sizeof(T);
  using WQ = typename Word<V>::type;
  const int lx = threadIdx.x & (g.LX - 1), j = threadIdx.x / g.LX;
  for (long long blk = blockIdx.x; blk < g.blocks; blk += gridDim.x) {
    const long long t = blk % g.px_tiles, rb = blk / g.px_tiles, b = rb / g.run_blocks;
    const long long run = (rb - b * g.run_blocks) * g.J + j;
    const int grp = (int)(run / g.per_group), in_group = (int)(run - (long long)grp * g.per_group), apart = SHIFT ? g.apart : 1;
    const int c0 = grp * a.G + in_group / apart * (apart * kRun) + in_group % apart;
    const int nc = run < g.runs ? max(0, min(kRun, (min((grp + 1) * a.G, a.C) - c0 + apart - 1) / apart)) : 0;
    const long long pos = t * g.TP, row0 = (b * a.C + c0) * a.P + pos, step = apart * a.P;
    const int n = (int)min((long long)g.TP, a.P - pos);  // pixels of the tile
    const int m = SHIFT ? (int)((unsigned)row0 & (V - 1)) : 0, px = lx * V - m;
    const long long s0 = (b * a.NG + grp) * a.P + pos + px;
    F<V> s = fill<V>(0.0f);
    WQ w[kRun];
    if constexpr (SHIFT) {
      if (nc > 0)
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (px + e >= 0 && px + e < n) s.v[e] = a.scale[s0 + e];
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        memset(&w[i], 0, sizeof(WQ));
        const long long at = row0 + i * step + px;
        if (i < nc && px < n && DISCO_IN_BOUNDS(at >= 0 && at < a.n)) {
          if (at + V <= a.n) {
            w[i] = load_stream<WQ>(a.q + at);
          } else {
            uint8_t z[V] = {};
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (at + e < a.n) z[e] = a.q[at + e];
            memcpy(&w[i], z, V);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        store_words<V>((T*)a.x + row0 + i * step - m, row0 + i * step - m, a.n, packed<T, V>(mul(unpack_e4m3<V>(w[i]), s)), m, lx, g.LX, n, i < nc);
    } else if (nc > 0 && px < n) {
      if (DISCO_IN_BOUNDS(s0 + V <= (long long)a.B * a.NG * a.P)) {
#pragma unroll
        for (int e = 0; e < V; e += 4) {
          const float4 f = *reinterpret_cast<const float4*>(a.scale + s0 + e);
          s.v[e] = f.x, s.v[e + 1] = f.y, s.v[e + 2] = f.z, s.v[e + 3] = f.w;
        }
      }
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (i < nc && DISCO_IN_BOUNDS(row0 + i * a.P + px + V <= a.n)) w[i] = load_stream<WQ>(a.q + row0 + i * a.P + px);
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (i < nc && DISCO_IN_BOUNDS(row0 + i * a.P + px + V <= a.n))
          store_stream((T*)a.x + row0 + i * a.P + px, packed<T, V>(mul(unpack_e4m3<V>(w[i]), s)));
    }
  }
}

// Rows of features (P = 1): words of V elements of the whole array.  ONE: V
// divides G and C, a word has one scale.
template <typename T, bool ONE>
__global__ void __launch_bounds__(kThreads) dequant_rows_kernel(const DequantArgs a) {
  constexpr int V = 16 / (int)sizeof(T);
  using WQ = typename Word<V>::type;
  const long long words = (a.n + V - 1) / V, stride = (long long)gridDim.x * kThreads;
  for (long long k0 = (long long)blockIdx.x * kThreads + threadIdx.x; k0 < words; k0 += 4 * stride) {
    WQ w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long at = (k0 + u * stride) * V;
      if (at + V <= a.n) w[u] = load_stream<WQ>(a.q + at);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const long long at = (k0 + u * stride) * V;
      if (at >= a.n) continue;
      long long b = a.n <= 0xffffffffLL ? (long long)((unsigned)at / (unsigned)a.C) : at / a.C;
      int c = (int)(at - b * a.C), grp = c / a.G;
      if (at + V <= a.n) {
        F<V> s;
        if constexpr (ONE) {
          s = fill<V>(a.scale[b * a.NG + grp]);
        } else {
          int end = min((grp + 1) * a.G, a.C);
          float z = a.scale[b * a.NG + grp];
#pragma unroll
          for (int e = 0; e < V; ++e, ++c) {
            if (c == end) {
              ++grp;
              if (c == a.C) c = 0, grp = 0, ++b;
              end = min((grp + 1) * a.G, a.C);
              z = a.scale[b * a.NG + grp];
            }
            s.v[e] = z;
          }
        }
        store_stream((T*)a.x + at, packed<T, V>(mul(unpack_e4m3<V>(w[u]), s)));
      } else {  // the array's last elements
        for (long long i = at; i < a.n; ++i) {
          const long long r = i / a.C;
          const __half v = __half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)a.q[i], __NV_E4M3));
          ((T*)a.x)[i] = from_f32<T>(__half2float(v) * a.scale[r * a.NG + (i - r * a.C) / a.G]);
        }
      }
    }
  }
}

template <typename T>
int dequant(const DequantArgs& a, cudaStream_t st) {
  constexpr int V = 16 / (int)sizeof(T);
  if (a.P == 1) {
    const long long words = (a.n + V - 1) / V;
    const int grid = (int)min((words + kThreads - 1) / kThreads, (long long)kSMs * 8);
    if (a.C % V == 0 && a.G % V == 0) dequant_rows_kernel<T, true><<<grid, kThreads, 0, st>>>(a);
    else dequant_rows_kernel<T, false><<<grid, kThreads, 0, st>>>(a);
    return check_launch("dequant_rows_kernel");
  }
  Cut g;
  g.apart = 1;
  while (a.P * g.apart % V) g.apart *= 2;
  const bool shifted = g.apart > 1;
  const int spare = shifted ? 1 : 0;
  const long long words = (a.P + V - 1) / V + spare;
  g.LX = 32;
  while (g.LX > 1 + spare && g.LX / 2 >= words) g.LX /= 2;
  g.J = kThreads / g.LX;
  g.TP = (g.LX - spare) * V;
  g.per_group = (a.G + kRun * g.apart - 1) / (kRun * g.apart) * g.apart;
  g.runs = (long long)a.NG * g.per_group;
  g.run_blocks = (g.runs + g.J - 1) / g.J;
  g.px_tiles = (a.P + g.TP - 1) / g.TP;
  g.blocks = a.B * g.run_blocks * g.px_tiles;
  const int grid = (int)min(g.blocks, 1LL << 30);
  if (shifted) dequant_kernel<T, true><<<grid, kThreads, 0, st>>>(a, g);
  else dequant_kernel<T, false><<<grid, kThreads, 0, st>>>(a, g);
  return check_launch("dequant_kernel");
}

}  // namespace
}  // namespace disco

using namespace disco;
using namespace disco::norm;

extern "C" int disco_dequant_e4m3(const void* q, const float* scale, void* x, int32_t group, int32_t B, int32_t C,
                                  int64_t P, disco_dtype dtype, void* stream) {
  disco::NvtxScope nvtx_scope("disco_dequant_e4m3");
  int rc;
  if ((rc = check_shape(B, C, P, dtype))) return rc;
  if (!q || !scale || !x) return fail(DISCO_ERR_INVALID_ARG, "q, scale or x is null");
  if (group < 0) return fail(DISCO_ERR_INVALID_ARG, "group must be >= 0");
  if ((rc = check_device())) return rc;
  DequantArgs a{(const uint8_t*)q, scale, x, 0, 0, B, C, P, (long long)B * C * P};
  a.NG = groups(C, group, &a.G);
  const Buffer in[] = {{q, (size_t)a.n, "q"}, {scale, (size_t)B * a.NG * P * 4, "scale"}};
  const Buffer out[] = {{x, (size_t)a.n * elem_bytes(dtype), "x"}};
  const unsigned in_place[] = {0, 0};
  if ((rc = check_buffers(in, in_place, 2, out, 1))) return rc;
  const cudaStream_t st = (cudaStream_t)stream;
#define CALL(T) rc = dequant<T>(a, st)
  DISCO_BY_DTYPE(dtype, CALL)
#undef CALL
  return rc;
}
