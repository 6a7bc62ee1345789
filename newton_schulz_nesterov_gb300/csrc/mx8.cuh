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

// Exponents are found from the high halves of magnitudes' bits, which do not fall
// as a magnitude grows: a block's parts are compared by them, two in a word.
// amax = 1.m x 2^(ex-127): floor takes ex - 8; 448 = 1.75 x 2^8, so ceil takes
// one more where 1.m > 1.75, which is where adding 0x1FFFFF to the bits carries
// into the exponent.  What is not finite is then put above every finite one.
struct Rounding {
  uint32_t up;      // added to the bits: 0 (floor), 0x1FFFFF (ceil)
  uint32_t not_finite;  // the least half of one that is not
};
__host__ __device__ constexpr Rounding rounding_of(bool ceil) { return ceil ? Rounding{0x1FFFFFu, 0xFFFFu} : Rounding{0u, 0x7F80u}; }
__device__ __forceinline__ uint32_t key_bits(float amax, const Rounding& r) {
  const uint32_t bits = __float_as_uint(amax);
  if (r.up == 0) return bits;
  return bits >= 0x7F800000u ? 0xFFFF0000u : bits + r.up;
}
// The keys of two magnitudes, the first in the low half.
__device__ __forceinline__ uint32_t keys2(float a, float b, const Rounding& r) { return __byte_perm(key_bits(a, r), key_bits(b, r), 0x7632); }
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }
__device__ __forceinline__ bool any_not_finite(uint32_t two, const Rounding& r) { return (two & 0xFFFFu) >= r.not_finite || (two >> 16) >= r.not_finite; }

// max(ex, 8) of a key; the scale byte is 8 less (255 where the key is not finite),
// and 2^(127 - byte) the factor of the block's values.
__device__ __forceinline__ uint32_t exponent_of(uint32_t two, int half) { return max(half ? two >> 23 : (two >> 7) & 0x1FFu, 8u); }
__device__ __forceinline__ uint32_t byte_of(uint32_t two, int half, const Rounding& r) {
  return (half ? two >> 16 : two & 0xFFFFu) >= r.not_finite ? 255u : exponent_of(two, half) - 8u;
}
__device__ __forceinline__ float factor_of(uint32_t exponent) { return __uint_as_float((262u - exponent) << 23); }

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
