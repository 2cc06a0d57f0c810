// Rows in groups of 32 values with a power of two each (the OCP microscaling
// formats MXFP8 and MXFP4): activations as e4m3 bytes, weights as e2m1 values,
// two to a byte, scales as bytes e + 127 in tiles of 128 rows x 4 groups --
// the arrangement that the block-scaled tensor-core products read, so a tile
// goes from memory to the scale columns of tensor memory as it lies.
//
// A group's scale is 2^e with the smallest e in [-126, 120] whose top * 2^e
// covers the group's largest magnitude (top: 448 for e4m3, 6 for e2m1), so the
// division by the scale is exact and no finite value saturates but weights beyond
// 6 * 2^120.
#pragma once

#include "s2_common.cuh"

namespace s2 {

constexpr int kMxEMin = -126, kMxEMax = 120;
constexpr int kMxTile = 512;      // bytes of a scale tile

// Byte of (row, 128-value column block kt) in scale tiles of KT column blocks:
// the word with the scales of its four groups.
__host__ __device__ inline size_t mx_scale_at(long long row, int kt, int KT) {
  return ((size_t)(row >> 7) * KT + kt) * kMxTile + (size_t)(row & 31) * 16 + ((row >> 5) & 3) * 4;
}

S2_DEV float mx_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }   // |e| <= 126
// 2^(b - 127) of a scale byte; 255 is NaN, 0 the subnormal 2^-127.
S2_DEV float mx_scale(uint32_t b) {
  return b == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(b ? b << 23 : 0x00400000u);
}
// The smallest e in range with amax <= 1.75 * 2^8 * 2^e, or 1.5 * 2^2 * 2^e.
S2_DEV int mx8_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return min(max((int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0), kMxEMin), kMxEMax);
}
S2_DEV int mx4_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  return min(max((int)(u >> 23) - 129 + ((u & 0x7fffffu) > 0x400000u ? 1 : 0), kMxEMin), kMxEMax);
}

// Two values to e4m3 / e2m1 (nearest, ties to even, saturating; NaN stays NaN
// in e4m3), x in the low byte / low four bits.
S2_DEV uint32_t mx_e4m3x2(float x, float y) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(y), "f"(x));
  return r;
}
S2_DEV uint32_t mx_e2m1x2(float x, float y) {
  uint32_t r;
  asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
      : "=r"(r) : "f"(y), "f"(x));
  return r;
}
S2_DEV float mx_e4m3(uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(b & 0xffu));
  float f;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.f32.f16 %0, l;\n\t}" : "=f"(f) : "r"(r));
  return f;
}

}  // namespace s2
