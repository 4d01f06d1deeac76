// int8 rows: codes with one scale per row (moe.h, "int8 experts"). A row of values v with a = max|v| has the codes
// round-half-even(127 v / a), where a tie is one of the quotient of the real numbers, and the scale a / 127.
#pragma once

#include "common.h"

namespace moe {

// What a row's codes need of its maximum. `top` is the largest bit pattern of the row's |v|: that of a NaN is above
// infinity's, so a row with either shows it here.
struct I8Row {
  float a, inv, pre;  // maximum and 127 / maximum after scaling by pre, a power of two that keeps both in range
  float scale;
  bool finite;
};
__device__ __forceinline__ I8Row i8_row(uint32_t top) {
  I8Row r;
  const float a = __uint_as_float(top);
  r.finite = top < 0x7f800000u;
  // an element that pre makes subnormal is below 2^-60 of the maximum: its code is 0 either way
  r.pre = a < 0x1p-60f ? 0x1p60f : a > 0x1p60f ? 0x1p-60f : 1.f;
  r.a = a * r.pre;
  r.inv = a > 0.f ? 127.f / r.a : 0.f;
  r.scale = r.finite ? a / 127.f : __uint_as_float(0x7fc00000u);
  return r;
}

// The code of v as a word whose low byte holds it. v * inv is within 2^-15 of 127 v / a, so adding 1.5 * 2^23, which
// rounds to whole numbers and leaves them in the low bits, gives the code unless the product is that near a tie; there
// the quotient is formed in double, where 127 v is exact and a quotient that is no tie does not round to one (it is at
// least 2^-25 / 128 of itself away). Dividing for every element instead makes the vector units the bound.
__device__ __forceinline__ uint32_t i8_code(float v, const I8Row& r) {
  const float t = v * r.pre * r.inv;
  float n = t + 12582912.f;
  if (fabsf(t - (n - 12582912.f)) > 0.5f - 0x1p-13f)
    n = (float)rint(127.0 * (double)(v * r.pre) / (double)r.a) + 12582912.f;
  return __float_as_uint(n);
}
__device__ __forceinline__ uint32_t i8_pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u), hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
  return lo | (hi << 16);
}
// The codes of N values, four to a word; zeros where the row is not finite.
template <int N>
__device__ __forceinline__ void i8_codes(const float (&v)[N], const I8Row& r, uint32_t (&w)[N / 4]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    w[i] = r.finite ? i8_pack4(i8_code(v[4 * i], r), i8_code(v[4 * i + 1], r), i8_code(v[4 * i + 2], r),
                               i8_code(v[4 * i + 3], r))
                    : 0u;
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
template <int N>
__device__ __forceinline__ uint32_t abs_top(const float (&v)[N], uint32_t top) {
#pragma unroll
  for (int i = 0; i < N; ++i) top = max(top, abs_bits(v[i]));
  return top;
}
__device__ __forceinline__ uint32_t wave_top(uint32_t top) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, off, 64));
  return top;
}

}  // namespace moe
