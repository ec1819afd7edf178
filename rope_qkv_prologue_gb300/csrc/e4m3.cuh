// e4m3 values of the 8-bit key/value pool: conversions and the scales' range.
#pragma once

#include <stdint.h>

namespace qkvp {

constexpr float kE4m3Max = 448.f;
// Scales lie between these; one outside is taken as the nearest (a NaN as the least).
constexpr float kScaleLeast = 7.888609052210118e-31f;  // 2^-100
constexpr float kScaleMost = 1.329227995784916e36f;    // 2^120

__device__ __forceinline__ float clamp_scale(float s) { return fminf(fmaxf(s, kScaleLeast), kScaleMost); }

// Two floats to two codes (round to nearest even, beyond 448 to 448), `lo` in the low byte.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  return to_e4m3x2(a, b) | (to_e4m3x2(c, d) << 16);
}

// Four codes to four values as two pairs of f16 (exact).
__device__ __forceinline__ void from_e4m3x4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

}  // namespace qkvp
