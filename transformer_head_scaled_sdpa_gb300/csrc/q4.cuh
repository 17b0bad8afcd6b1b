// q4.cuh -- the 4-bit cache's format: how a row is quantised and read.
#pragma once

#include <cstdint>

#include "fp8.cuh"
#include "ptx.cuh"

namespace mha {

// A row x of the 4-bit cache is kept as codes c = 0 .. 15 and two bf16 numbers, its
// offset lo = min x and its step, and stands for lo + c * step:
//     step = the smallest bf16 s with lo + 15 s >= max x, s >= 2^-13 max |x|, s >= 2^-60
//     c    = the integer nearest to (x - lo) / step, a tie to the lower one
// Both are decided exactly (lo is an input value, bf16 numbers compare exactly with the
// directed roundings of a fused multiply-add), so that the codes follow from the
// definition alone.  The bound 2^-13 max |x| binds only for rows of one value (the
// spacing of bf16 values is at least 2^-8 of the smaller one, over 15): it keeps lo /
// step, which the attention sums, inside float32.  A row that holds a NaN or an
// infinity, or whose spread passes float32's range, has lo = NaN and reads as NaN.
// Two codes to a byte, feature 2 i in the low four bits of byte i.
constexpr float kMinStep = 8.67361738e-19f;  // 2^-60

struct RowQ4 {
  float lo, step;
  float inv;     // a little below 1 / step
  bool careful;  // codes_q4 has to look twice
};

// The row's offset and step from its smallest and largest value.
__device__ __forceinline__ RowQ4 row_q4(float lo, float hi) {
  RowQ4 r;
  const float spread = hi - lo;
  if (!(spread < INFINITY)) {
    r.lo = __int_as_float(0x7fc00000);
    r.step = kMinStep;
    r.inv = 0.f;
    r.careful = false;
    return r;
  }
  r.lo = lo + 0.f;  // (-0 as 0)
  // a bf16 number below the one wanted, by one or two steps
  float s = __uint_as_float(__float_as_uint(spread * 0.0666666f) & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (!(__fmaf_rd(15.f, s, lo) >= hi)) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
  r.step = fmaxf(fmaxf(s, fmaxf(fabsf(lo), fabsf(hi)) * 0x1p-13f), kMinStep);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(r.step));  // (to 2^-23)
  r.inv = inv * (1.f - 0x1p-20f);
  const float zero = -r.lo * inv, part = zero - floorf(zero);
  r.careful = (r.lo != 0.f && fabsf(r.lo) < 0.0148f * r.step) || fabsf(part - 0.5f) < 0.0149f;
  return r;
}

constexpr float kToInteger = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer

// A value's code, whatever the row.  The first estimate is the code or the one above (its
// factor is a little too large); x at or below the middle between it and the one below
// takes that.
__device__ __forceinline__ uint32_t code_q4(float x, const RowQ4& r) {
  const float up = fmaf(x - r.lo, r.inv * (1.f + 0x1p-17f), kToInteger);
  const uint32_t c = __float_as_uint(up) & 15u;
  return x > __fmaf_rd(up - kToInteger - 0.5f, r.step, r.lo) ? c : c - 1u;
}

// The codes of eight values, four bits each, the first in the lowest.  For nearly all rows
// one rounded product decides.  q = (x - lo) / step against a middle h = k + 1/2: where
// they differ, by u / (2 step) at least, u the last place of x, of lo or half of step's,
// whichever is finest; relative to q, u / (2 (x - lo)).  Where |x| and |lo| are at least
// 2^-10 (x - lo) (or lo is 0) that is 2^-19 or more, while the product is below q by 2^-20
// with an error of 2^-21.6: it lies on q's side of h, and below h when q = h.  Else q is
// within 15 * 2^-10 of -lo / step (x near 0), or lo is that near 0: rows where -lo / step
// is that near to a middle, or to 0, are `careful`.
__device__ __forceinline__ uint32_t codes_q4(const float (&x)[8], const RowQ4& r) {
  uint32_t c = 0;
  if (r.careful) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c |= code_q4(x[i], r) << (4 * i);
    return c;
  }
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    float a, b;
    add2(a, b, x[i], x[i + 1], -r.lo, -r.lo);
    fma2(a, b, a, b, r.inv, r.inv, kToInteger, kToInteger);
    c = (c * 16u + __float_as_uint(b)) * 16u + __float_as_uint(a);
  }
  return c - 0x4b400000u * 0x11111111u;  // (less kToInteger's bits in every place)
}

}  // namespace mha
