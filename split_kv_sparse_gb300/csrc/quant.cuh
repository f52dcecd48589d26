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
// zero keeps q's sign). Where y is not a normal number, or a q leaves the range, the
// eight values are divided one by one (in a loop of its own: sixteen divisions
// inlined here cost 24.2 us where this takes 20.1, 16,001 rows of 8 heads into e4m3).
struct Divider {
  float d, y;
  bool plain;
};
__device__ __forceinline__ Divider divider(float d) {
  Divider by;
  by.d = d;
  by.y = __fdiv_rn(1.f, d);
  by.plain = !(fabsf(by.y) >= 1.17549435e-38f && fabsf(by.y) <= 3.40282347e38f);
  return by;
}
__device__ __forceinline__ float quotient(float x, float d, float y) {
  const float q = __fmul_rn(x, y);
  return copysignf(__fmaf_rn(__fmaf_rn(-q, d, x), y, q), q);
}
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
// x = x / d, eight values.
__device__ __forceinline__ void divide8(float (&x)[8], const Divider& by) {
  float q[8], most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    most = fmaxf(most, fabsf(__fmul_rn(x[i], by.y)));
    q[i] = quotient(x[i], by.d, by.y);
  }
  if (by.plain || most > 1e30f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v = i == k ? x[k] : v;
      v = __fdiv_rn(v, by.d);
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = i == k ? v : q[k];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = q[i];
}

// max(a, |x|) that keeps a NaN of either.
__device__ __forceinline__ float max_abs_nan(float a, float x) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(x)));
  return r;
}

// The scale of 16 dims whose largest magnitude (after the descale) is amax: e4m3(amax / 6), which takes the largest of
// them to e2m1's largest value. A NaN among them makes the scale NaN, as e2m1 has none.
__device__ __forceinline__ uint32_t scale_code(float amax) { return e4m3x2(__fdiv_rn(amax, 6.f), 0.f) & 0xffu; }
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t h;
  asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(code));
  float f;
  asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.f32.f16 %0, lo;\n}\n" : "=f"(f) : "r"(h));
  return f;
}
// The e2m1 codes of eight y / scale (ties to even, at most 6), the first in the lowest four bits. The quotient is the
// rounded one, as e2m1 of a division. Where the scale is 0 or NaN every code is a zero with its value's sign. (Beyond
// 6 * 448 every code is the largest; the clamp keeps infinities out of the quotient's residual.)
__device__ __forceinline__ uint32_t e2m1x8(const float (&y)[8], float scale) {
  const float r = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float q[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float v = fminf(fmaxf(y[2 * i + k], -4096.f), 4096.f);
      q[k] = scale > 0.f ? quotient(v, scale, r) : copysignf(0.f, y[2 * i + k]);
    }
    uint32_t c;
    asm("{\n  .reg .b8 b;\n  cvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n  cvt.u32.u8 %0, b;\n}\n" : "=r"(c) : "f"(q[0]), "f"(q[1]));
    w |= c << (8 * i);
  }
  return w;
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
// Two e4m3 codes (the low half of w) as an f16 pair (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t w) {
  uint32_t h;
  asm("{\n  .reg .b16 lo, hi;\n  mov.b32 {lo, hi}, %1;\n  cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(h) : "r"(w));
  return h;
}

}  // namespace skv
