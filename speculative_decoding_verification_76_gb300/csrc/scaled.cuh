// The scales of a scaled cache (e4m3 codes with one scale for each block of tokens and KV head),
// shared by the calls that write one (append_scaled.cu).
//
// Why powers of two: e4m3 is a floating-point type, so any scale that keeps the largest value
// below 448 gives the same relative precision; a power of two makes a block's codes move to a
// larger scale exactly (but for what falls below the type's normal numbers), so that a block can
// be filled token by token without rounding its first tokens again and again, and makes the
// stored value the rounded x itself, whatever the scale.
#pragma once
#include <cuda_fp16.h>

#include "serving.cuh"

constexpr int kMaxBlock = 64;
constexpr float kLeastScale = 0x1p-64f;

// The smallest 2^k >= 2^-64 with x <= 448 * 2^k (448 = 1.75 * 2^8), x >= 0 and finite.
SPEC_DEV float needed_scale(float x) {
  const uint32_t u = __float_as_uint(x);
  const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  return __uint_as_float((uint32_t)max(e, 127 - 64) << 23);
}

// What a stored scale counts as beside it: the next power of two; 0 if it is not positive and
// finite.
SPEC_DEV float held_scale(float s) {
  if (!(s > 0.f) || s == INFINITY) return 0.f;
  const uint32_t u = __float_as_uint(s) + 0x7fffffu;
  return __uint_as_float(min(u, 0x7f000000u) & 0x7f800000u);
}

SPEC_DEV uint32_t e4m3_word(float x0, float x1, float x2, float x3) {  // nearest even, +-448
  uint32_t r;
  asm("{\n .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n"
      " cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n mov.b32 %0, {lo, hi};\n}\n"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

SPEC_DEV void e4m3_values(uint32_t w, float* x) {  // of the four bytes
  uint32_t lo, hi;
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n"
      " cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}

// 16 codes under another scale: times the ratio of the old one to the new.
SPEC_DEV uint4 moved_codes(uint4 w, float ratio) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x[4];
    e4m3_values(u[i], x);
    u[i] = e4m3_word(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
  }
  return w;
}

// |x|, if it is finite (what is not does not count for a scale)
SPEC_DEV float finite_abs(float x) {
  const float y = fabsf(x);
  return y < INFINITY ? y : 0.f;
}
