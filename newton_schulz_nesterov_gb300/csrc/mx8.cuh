// MXFP8 on the device: a block's scale byte, codes and values.
//
// Block of 32 elements, amax = max |x|:
//   floor  e = floor(log2 amax) - 8     ceil  e = least with amax <= 448 2^e
//   (not below -127; amax = 0: -127), scale byte e + 127
//   code = E4M3 of x 2^-e, nearest, ties to the even code, saturating at 448
//   amax Inf or NaN: scale byte 255 (NaN), codes 0
// 2^-e is a power of two, so the scaled value is exact in fp32 and the codes
// do not depend on how it is computed.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace dmuon {
namespace mx8 {

// Larger magnitude of three, NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int N>
__device__ __forceinline__ float max_abs(const float (&v)[N]) {
  static_assert(N % 2 == 0, "pairs");
  float m = max_abs(0.f, v[0], v[1]);
#pragma unroll
  for (int i = 2; i < N; i += 2) m = max_abs(m, v[i], v[i + 1]);
  return m;
}

// Exponents are found from the high halves of magnitudes' bits ("keys"), which do
// not fall as a magnitude grows: a block's parts are compared by them, two in a
// word.  amax = 1.m x 2^(ex-127): floor takes ex - 8; 448 = 1.75 x 2^8, so ceil
// takes one more where 1.m > 1.75, which is where adding 0x1FFFFF to the bits
// carries into the exponent.  Keys of what is not finite are 0x7F80 or more, as
// ceil's of magnitudes above 1.75 x 2^127 are: those are then looked at again.
constexpr uint32_t kFloor = 0u, kCeil = 0x1FFFFFu;
__device__ __forceinline__ uint32_t keys2(float a, float b, uint32_t up) {  // the first in the low half
  return __byte_perm(__float_as_uint(a) + up, __float_as_uint(b) + up, 0x7632);
}
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
__device__ __forceinline__ bool may_not_be_finite(uint32_t two) { return (two & 0xFFFFu) >= 0x7F80u || two >= 0x7F800000u; }
__device__ __forceinline__ bool not_finite(float amax) { return __float_as_uint(amax) >= 0x7F800000u; }

// The exponents of two keys where they stand in an fp32's high half, not below 8:
// the scale byte is 8 less (255 for a block that is not finite), 2^(127 - byte)
// the factor of the block's values.
__device__ __forceinline__ uint32_t exponents2(uint32_t two) { return __vmaxu2(two, 0x04000400u) & 0xFF80FF80u; }
__device__ __forceinline__ uint32_t byte_of(uint32_t exponents, int half) { return (half ? exponents >> 23 : (exponents >> 7) & 0x1FFu) - 8u; }
__device__ __forceinline__ float2 factors2(uint32_t exponents) {  // (262 - exponent) << 23
  const uint32_t f = 0x83008300u - exponents;
  return make_float2(__uint_as_float(f << 16), __uint_as_float(f & 0xFFFF0000u));
}

// Four scaled values to four codes, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t w;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// Two codes (the low half of w) as fp32; exact.
__device__ __forceinline__ float2 values2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(w));
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}

// 2^(byte - 127), NaN for byte 255.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : (byte == 0u ? 0x00400000u : byte << 23));
}

}  // namespace mx8
}  // namespace dmuon
