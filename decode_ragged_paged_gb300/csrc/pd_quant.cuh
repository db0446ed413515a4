// pd_quant.cuh -- the 8-bit values of a quantized cache (e4m3: a sign, 4 bits of
// exponent, 3 of mantissa; largest 448, smallest step 2^-9, one NaN a sign and no
// infinities) and the scale of a block of them.
#pragma once

#include "pd_common.cuh"

namespace pd {

// Two fp32 values, of at most 448 or NaN, rounded to e4m3 (nearest, ties to even), `lo` in the low byte.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two e4m3 values (the low 16 bits) as fp32, exactly: through fp16, which holds all of them.
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
  float2 f;
  asm("{\n\t.reg .b32 h;\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.f16x2.e4m3x2 h, %2;\n\tmov.b32 {a, b}, h;\n\t"
      "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "h"((uint16_t)v));
  return f;
}

// Two times two e4m3 values, as two and two fp16 pairs, exactly: of a's low and high half, then b's.
__device__ __forceinline__ void pairs_to_f16(uint32_t a, uint32_t b, uint32_t (&out)[4]) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(out[0]), "=r"(out[1])
      : "r"(a));
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(out[2]), "=r"(out[3])
      : "r"(b));
}

// 16 e4m3 values as fp16, exactly.
__device__ __forceinline__ void to_f16(const uint4& v, uint32_t (&out)[8]) {
  uint32_t lo[4], hi[4];
  pairs_to_f16(v.x, v.y, lo);
  pairs_to_f16(v.z, v.w, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = lo[i], out[4 + i] = hi[i];
}

// log2 of a normal positive number with the hardware approximation.
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / b of a scale of V, given as log2 b: also above 2^126, where it is subnormal.
__device__ __forceinline__ float inverse_scale(float log_b) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(-log_b));
  return y;
}

// The softmax's sum is that of weights over their keys' scales of V. A row's largest weight is 2^3 or more and a scale
// below 2^128, so the sum is above 2^-125. At the other end scales are 2^-100 or more and all weights of a row of 2^24
// keys come to 2^36: more than fp32 holds. So where a sum has passed kSumHigh, it is held times kSumFactor from
// there on, below 2^112 with all that may still come, and with a minus sign where others have to tell.
constexpr float kSumHigh = 0x1p112f, kSumFactor = 0x1p-24f, kSumLog = 24.0f;

// The exponent of the scale of values up to amax (finite, not negative): the smallest power of two,
// at least 2^-100, times 448 is not below amax. 448 = 1.75 * 2^8. A power of two, because values
// are then scaled without rounding, and what a block holds already keeps its value when the scale grows
// (but for what falls below e4m3's smallest step); a scale of amax / 448 would be up to 2x smaller, which
// gives a floating type one binade more below and no bit.
__device__ __forceinline__ int scale_exponent(float amax) {
  const uint32_t bits = __float_as_uint(amax);
  const int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -100);
}

constexpr float kScaleMin = 0x1p-100f;  // the smallest scale

// 2^e, -126 <= e <= 127.
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

}  // namespace pd
