// fp8.cuh -- conversions between float32 / bf16 and the 8-bit formats, and the
// power-of-two scale of a row in the 8-bit cache.
#pragma once

#include <cstdint>

namespace mha {

// A row x of the 8-bit cache is kept as e4m3 codes c and one byte s with
// x = c * 2^(s - 127): e = s - 127 is the smallest integer >= kMinExponent
// with max |x| <= 448 * 2^e (448: the largest e4m3 value).  The scale is a
// power of two, so quantising rounds once (x * 2^-e is exact in float32) and
// reading back is exact; e4m3 being a floating format, a scale of 448 / max
// |x| would buy no precision but in its subnormals, 2^-17 and less of the
// row's largest value.
constexpr int kMinExponent = -64;
constexpr float kF8Max = 448.f;

// 2^e as a float, -126 <= e <= 127
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Biased exponent s of a row whose largest magnitude is amax (>= 0, not NaN;
// infinity gives 2^120).  amax = m 2^E with 1 <= m < 2 and 448 = 1.75 * 2^8,
// so e = E - 8, one more when m > 1.75.
__device__ __forceinline__ int row_scale_byte(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int E = static_cast<int>(bits >> 23) - 127;  // below -126: the clamp decides
  const int e = E - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (e < kMinExponent ? kMinExponent : e) + 127;
}

// Two floats to two codes (round to nearest even, saturating, NaN kept); lo in
// bits 0-7.
__device__ __forceinline__ uint16_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 codes to packed fp16 (exact); code in bits 0-7 to the low half.
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}

__device__ __forceinline__ float half_lo(uint32_t h2) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(h2));
  return f;
}
__device__ __forceinline__ float half_hi(uint32_t h2) {
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, h;\n\t}" : "=f"(f) : "r"(h2));
  return f;
}

// bf16 pairs -> float
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace mha
