// Number formats of the paged cache: exact fp32 division by one divisor, e4m3 codes, and the 4-bit form (e2m1 codes,
// an e4m3 scale for each 16 dims).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "softmax_util.cuh"

namespace skv {

// x / d for many x by one d, rounded to nearest as a division: with y = RN(1 / d) and q =
// RN(x y), the residual x - q d is exact in an FMA and q + (x - q d) y rounds to the quotient
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000", 1990; a
// zero keeps q's sign). The residual has to be a multiple of 2^-149: with d from 2^-90 up it is one for every q that a code
// tells from 0 (2^-11 and more, 24 bits each). Below that (a descale of 2^-116 gave codes one off), where y is not a
// normal number, or where a q leaves the range, the values are divided one by one, those of divide4 in a function of its own,
// the eight that pages.cu takes at a time in a loop (sixteen divisions inlined there cost 24.2 us where this takes 20.1, 16,001 rows
// of 8 heads into e4m3).
struct Divider {
  float d, y;
  bool plain;
};
__device__ __forceinline__ Divider divider(float d) {
  Divider by;
  by.d = d;
  by.y = __fdiv_rn(1.f, d);
  by.plain = !(fabsf(by.y) >= 1.17549435e-38f && fabsf(by.y) <= 0x1p90f);
  return by;
}
__device__ __forceinline__ float quotient(float x, float d, float y) {
  const float q = __fmul_rn(x, y);
  return copysignf(__fmaf_rn(__fmaf_rn(-q, d, x), y, q), q);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// x / d by divisions, where a quotient leaves the range that the short way is good for (a function of its own, which keeps
// the others' code short).
static __device__ __noinline__ float4 divide4_far(float4 x, float d) {
  return make_float4(__fdiv_rn(x.x, d), __fdiv_rn(x.y, d), __fdiv_rn(x.z, d), __fdiv_rn(x.w, d));
}
// x = x / d, four values.
__device__ __forceinline__ void divide4(float (&x)[4], const Divider& by) {
  float q[4], most = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    q[i] = quotient(x[i], by.d, by.y);
    most = fmaxf(most, fabsf(__fmul_rn(x[i], by.y)));
  }
  if (by.plain || most > 1e30f) {
    const float4 v = divide4_far(make_float4(x[0], x[1], x[2], x[3]), by.d);
    q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = q[i];
}

// max(a, |x|) that keeps a NaN of either.
__device__ __forceinline__ float max_abs_nan(float a, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(x)));
  return r;
}

// The scale of 16 dims whose largest magnitude (after the descale) is amax: e4m3(amax / 6), which takes the largest of
// them to e2m1's largest value. A NaN among them makes the scale NaN, as e2m1 has none. (Past 448 * 6 every scale is 448.)
__device__ __forceinline__ uint32_t scale_code(float amax) {
  const float q = quotient(fminf(amax, 1e6f), 6.f, 0.166666671633720397949f);   // RN(1 / 6)
  return e4m3x2(amax == amax ? q : amax, 0.f) & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(code));
  float f;
  asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.f32.f16 %0, lo;\n}\n" : "=f"(f) : "r"(h));
  return f;
}
// RN(1 / s) of an e4m3 value s > 0: one Newton step in FMAs takes every approximation within 1 ulp there (tried for all 126).
__device__ __forceinline__ float reciprocal_e4m3(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return __fmaf_rn(__fmaf_rn(-s, r, 1.f), r, r);
}
// The e2m1 codes of eight y / scale (ties to even, at most 6), the first in the lowest four bits; |y| <= 1e30. The quotient is
// the rounded one, as e2m1 of a division. Where the scale is 0 or NaN every code is a zero with its value's sign.
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[2][4], float scale) {
  // (the quotient by a reciprocal of 0 is a zero of y's sign)
  const bool some = scale > 0.f;
  const float r = some ? reciprocal_e4m3(scale) : 0.f, d = some ? scale : 0.f;
  uint32_t c;
  asm("{\n  .reg .b8 b0, b1, b2, b3;\n  cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n  cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
      "  cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n  mov.b32 %0, {b0, b1, b2, b3};\n}\n"
      : "=r"(c)
      : "f"(quotient(y[0][0], d, r)), "f"(quotient(y[0][1], d, r)), "f"(quotient(y[0][2], d, r)), "f"(quotient(y[0][3], d, r)),
        "f"(quotient(y[1][0], d, r)), "f"(quotient(y[1][1], d, r)), "f"(quotient(y[1][2], d, r)), "f"(quotient(y[1][3], d, r)));
  return c;
}
// Eight e2m1 codes as four f16 pairs (exact).
__device__ __forceinline__ void f16_of_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n  .reg .b8 b0, b1, b2, b3;\n  mov.b32 {b0, b1, b2, b3}, %4;\n"
      "  cvt.rn.f16x2.e2m1x2 %0, b0;\n  cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      "  cvt.rn.f16x2.e2m1x2 %2, b2;\n  cvt.rn.f16x2.e2m1x2 %3, b3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A bf16 row of Q in f16 beside 4-bit pages: times 2^(141 - e) with e the exponent field of its largest element, which comes to lie in
// [2^14, 2^15) (rows below 2^-113 times 2^127), so the row is exact down to 2^-28 of that element and smaller ones are off by 2^-39
// of it at most. The second factor undoes the first.
__device__ __forceinline__ float f16_row_up(int e) { return __int_as_float(min(268 - e, 254) << 23); }
__device__ __forceinline__ float f16_row_down(int e) { return e > 14 ? __int_as_float((e - 14) << 23) : __int_as_float(1 << 22); }

// Two e4m3 codes (the low half of w) as an f16 pair (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t w) {
  uint32_t h;
  asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(w));
  return h;
}

}  // namespace skv
