// disco_i8.cuh -- what the operators on 8-bit integer activations share: the
// magnitudes and the rounding of a token's 8-bit form (disco_tokens.cuh), and how
// the integer products are described (disco_i8_mm.cuh).  Not part of the ABI.
//
// A token is one pixel of one sample (P = 1: one row of features).  Its 8-bit form:
//   a = max(1e-30, max_c |x_c|),  scale = a / 127,  q_c = round(127 x_c / a)
#pragma once

#include "disco_norm.cuh"

namespace disco {
namespace i8 {

using norm::check_buffers;
using norm::check_shape;
using norm::Buffer;
using norm::elem_bytes;
using norm::kSMs;

constexpr float kQMax = 127.0f;
constexpr float kAmaxFloor = 1e-30f;

// The largest magnitude as the bits of |x|: integers order them like the values,
// infinities above all finite ones and NaN above infinities, so a NaN is kept.
__device__ __forceinline__ uint32_t max16(uint32_t m, uint32_t w) { return __vmaxu2(m, w & 0x7fff7fffu); }
__device__ __forceinline__ uint32_t max32(uint32_t m, uint32_t w) { return max(m, w & 0x7fffffffu); }

// What a token's values are multiplied by.  For 16-bit inputs the quotient
// 127 x / a is rounded correctly: k x is exact (11 + 7 bits), inv is the correctly
// rounded reciprocal of b = a f (f a power of two that keeps all steps within
// fp32's normal range), and one remainder step t + (k x - t b) inv then gives
// the correctly rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990).  A
// quotient that is not half of an odd integer lies further from one than fp32's
// rounding moves it (2^-19 against 2^-24 relative), so q is the definition's, ties included.
struct Quantizer {
  float k, b, inv, scale;
  __device__ __forceinline__ explicit Quantizer(float amax) {  // amax >= 0, or infinite or NaN
    const float a = amax < kAmaxFloor ? kAmaxFloor : amax;     // keeps NaN
    const float f = a > 1e30f ? 0x1p-64f : a < 1e-20f ? 0x1p64f : 1.0f;
    b = a * f;
    k = kQMax * f;
    inv = __frcp_rn(b);
    scale = a / kQMax;
  }
};

// round(t) of |t| < 2^22, to nearest even, as the low bits of a float's pattern
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23

// The low byte of the result is q of one value of a token.
template <typename T>
__device__ __forceinline__ uint32_t quantize(float x, const Quantizer& z) {
  const float kx = z.k * x;
  float t = kx * z.inv;
  t = fmaf(fmaf(-t, z.b, kx), z.inv, t);
  if (!(fabsf(t) < 128.0f)) t = 0.0f;  // a token with an infinity or a NaN: its scale says so
  return __float_as_uint(t + kRound);
}
// fp32 inputs: 127 x takes 31 bits.  Within 2^-14 of a border (the error of t is
// below 2^-15) the quotient is taken in 64 bits, where it cannot reach the wrong side.
template <>
__device__ __forceinline__ uint32_t quantize<float>(float x, const Quantizer& z) {
  float t = (z.k * x) * z.inv;
  if (!(fabsf(t) < 128.0f)) t = 0.0f;
  const float r = (t + kRound) - kRound;
  if (fabsf(fabsf(t - r) - 0.5f) < 0x1p-14f) t = (float)rint((double)z.k * (double)x / (double)z.b);
  return __float_as_uint(t + kRound);
}

__device__ __forceinline__ uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The same for the gated activation y, in fp32.  For tensors of 16 bits within a few units
// of 2^-24 of the quotient; of 32 bits by the formula's own steps, each rounded correctly.
// Next to the middle of two integers either may come out.
template <typename T>
__device__ __forceinline__ uint32_t quantize_y(float y, const Quantizer& z) {
  const float ky = __fmul_rn(z.k, y);
  float t = sizeof(T) == 4 ? __fdiv_rn(ky, z.b) : ky * z.inv;
  if (!(fabsf(t) < 128.0f)) t = 0.0f;
  return __float_as_uint(t + kRound);
}

// act(g) and act'(g).  SiLU: g s, s (1 + g (1 - s)) with s = 1 / (1 + e^-g).
// GELU: g Phi, Phi + g phi with the normal distribution Phi and its density phi.
// T: the tensors' type.  16-bit ones take the approximate exponential and reciprocal of
// t = e^-|g|, s = (1 or t) / (1 + t): 2^-22 of the exponential, 2^-23 |g| of its argument's
// rounding, 2^-23 of the reciprocal and 2^-24 of each sum and product, within 2^-20 + 2^-23 |g| together,
// below the types' rounding of 2^-8 or 2^-11; gates below -87 give 0.
template <typename T>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(T) == 4) return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-g)));
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(-1.44269504f * fabsf(g)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
  return (g < 0.0f ? t : 1.0f) * r;
}
template <typename T, int V>
__device__ __forceinline__ norm::F<V> gated(const norm::F<V>& g, const norm::F<V>& v, int kind) {
  norm::F<V> y;
  if (kind == DISCO_GELU) {
#pragma unroll
    for (int e = 0; e < V; ++e) y.v[e] = __fmul_rn(__fmul_rn(g.v[e], __fmul_rn(0.5f, erfcf(-0.70710678f * g.v[e]))), v.v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) y.v[e] = __fmul_rn(__fmul_rn(g.v[e], sigmoid<T>(g.v[e])), v.v[e]);
  }
  return y;
}
template <typename T>
__device__ __forceinline__ float act_grad(float g, int kind, float* value) {
  if (kind == DISCO_GELU) {
    const float cdf = 0.5f * erfcf(-0.70710678f * g);
    *value = g * cdf;
    return fmaf(0.39894228f * g, sizeof(T) == 4 ? expf(-0.5f * g * g) : __expf(-0.5f * g * g), cdf);
  }
  const float s = sigmoid<T>(g);
  *value = g * s;
  return s * fmaf(g, 1.0f - s, 1.0f);
}

// The larger of m and |v|, NaN where one is.
__device__ __forceinline__ float max_abs(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// The float that a byte of a word of 8-bit integers stands for (E = 0 .. 3), exactly.
__device__ __forceinline__ float from_byte(uint32_t flipped, int e) {  // flipped: word ^ 0x80808080
  return __uint_as_float(__byte_perm(flipped, 0x4b000000u, 0x7440 + e)) - 8388736.0f;
}

// The nb bytes from byte sh of two words on, zeros behind them.
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int sh, int nb) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (sh & 8)
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  if (sh & 4)
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[i], w[i + 1], 8 * (sh & 3));
  if (nb < 16)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int left = nb - 4 * i;  // bytes of this word that belong to the line
      if (left < 4) o[i] = left <= 0 ? 0 : o[i] & (0xffffffffu >> (32 - 8 * left));
    }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace i8
}  // namespace disco
