// q4.cuh -- the 4-bit cache's format: how a row is quantised and read.
#pragma once

#include <cstdint>

#include "fp8.cuh"

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
  float lo, step, inv;  // (inv: a little above 1 / step)
};

// The row's offset and step from its smallest and largest value.
__device__ __forceinline__ RowQ4 row_q4(float lo, float hi) {
  RowQ4 r;
  const float spread = hi - lo;
  if (!(spread < INFINITY)) {
    r.lo = __int_as_float(0x7fc00000);
    r.step = kMinStep;
    r.inv = 0.f;
    return r;
  }
  r.lo = lo + 0.f;  // (-0 as 0)
  // a bf16 number below the one wanted, by one or two steps
  float s = __uint_as_float(__float_as_uint(spread * 0.0666666f) & 0xffff0000u);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (!(__fmaf_rd(15.f, s, lo) >= hi)) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
  r.step = fmaxf(fmaxf(s, fmaxf(fabsf(lo), fabsf(hi)) * 0x1p-13f), kMinStep);
  r.inv = __frcp_rn(r.step) * 1.000004f;
  return r;
}

// A value's code.  The first estimate is the code or the one above (its factor is a
// little too large); x at or below the middle between it and the one below takes that.
__device__ __forceinline__ uint32_t code_q4(float x, const RowQ4& r) {
  constexpr float kRound = 12582912.f;  // 1.5 * 2^23: adding it rounds to an integer
  const float up = fmaf(x - r.lo, r.inv, kRound);
  const float k = up - kRound;
  const uint32_t c = __float_as_uint(up) & 15u;
  return x > __fmaf_rd(k - 0.5f, r.step, r.lo) ? c : c - 1u;
}

}  // namespace mha
