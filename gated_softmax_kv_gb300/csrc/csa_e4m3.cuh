// e4m3 values (8 bits: sign, 4 exponent bits with bias 7, 3 mantissa bits;
// 0x7F and 0xFF are NaN) and the cache's power-of-two scales.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace csa {

constexpr int kScaleExpMin = -120, kScaleExpMax = 120;

// Two e4m3 values (low byte first) as fp16x2; exact, NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
  return r;
}

// Two fp32 values -> e4m3x2 (lo in the low byte), nearest even, finite values
// beyond 448 saturate, NaN gives 0x7F.
__device__ __forceinline__ uint32_t e4m3x2_of(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t e4m3x4_of(float a, float b, float c, float d) {
  return e4m3x2_of(a, b) | (e4m3x2_of(c, d) << 16);
}

__device__ __forceinline__ void e4m3x4_to_f32(uint32_t w, float* v) {
  const uint32_t a = e4m3x2_to_f16x2((uint16_t)(w & 0xFFFFu));
  const uint32_t b = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v[0]), "=f"(v[1])
      : "r"(a));
  asm("{\n\t.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(v[2]), "=f"(v[3])
      : "r"(b));
}

// 2^k as fp32, k in [-126, 127].
__device__ __forceinline__ float exp2i(int k) { return __int_as_float((k + 127) << 23); }

// The smallest k in [kScaleExpMin, kScaleExpMax] with amax <= 448 * 2^k, for
// finite amax >= 0: 448 = 1.75 * 2^8, so k is amax's exponent - 8, plus one
// where its significand is above 1.75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int k = (int)(b >> 23) - 127 - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(k, kScaleExpMin), kScaleExpMax);
}

}  // namespace csa
