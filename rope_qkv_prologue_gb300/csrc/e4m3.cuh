// e4m3 values of the 8-bit key/value pool: conversions and the scales' range.
#pragma once

#include <stdint.h>

namespace qkvp {

constexpr float kE4m3Max = 448.f;
// Scales lie between these; one outside is taken as the nearest (a NaN as the least). A block
// that grows by powers of two to hold values of up to 2^128 has a scale below 2^129 / 448,
// 1.15 2^120: below the bound, so that every scale that is written is read as it is.
constexpr float kScaleLeast = 0x1p-100f;
constexpr float kScaleMost = 0x1p121f;

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
