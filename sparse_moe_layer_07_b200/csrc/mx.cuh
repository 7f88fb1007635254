// Microscaled floating point: blocks of 32 values under one power-of-two scale
// (a byte e + 127, 255 = NaN), elements e2m1 (0, .5, 1, 1.5, 2, 3, 4, 6 and
// sign) for weights and e4m3 for activations.
//
// Scale of a block with largest magnitude m: 2^x with x = floor(log2 m) - emax
// (emax = 2 for e2m1, 8 for e4m3), one more when m is over 1.75 * 2^floor(log2 m):
// the largest element is then at most 7 (e2m1, rounds to 6) or 448 (e4m3, its
// largest value) in units of the scale, so an e4m3 element is never cut off and
// an e2m1 element loses at most 1/7; without the extra step it would lose up to
// 1/4.  x is kept within [-127, top]; a block that holds a NaN or an infinity
// gets the scale NaN.
//
// Scales are stored as the tensor core takes them: 512-byte blocks of 128 rows
// x 128 K, the byte of row r and 32-block k of the block at (r % 32) * 16 +
// (r / 32) * 4 + k.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kMxTopE2m1 = 125;  // 6 * 2^125 is finite in fp32 and bf16
constexpr int kMxTopE4m3 = 127;

// Exponent x of the scale from the bits of the largest magnitude.
template <int kEmax, int kTop>
__device__ __forceinline__ int mx_exponent(uint32_t amax_bits) {
  const int x = (int)(amax_bits >> 23) - 127 - kEmax + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return x < -127 ? -127 : (x > kTop ? kTop : x);
}

// 2^-x for x in [-127, 126].
__device__ __forceinline__ float mx_inverse(int x) { return __uint_as_float((uint32_t)(127 - x) << 23); }

__device__ __forceinline__ int mx_scale_at(int row, int kblock) {
  return (row & 31) * 16 + ((row & 127) >> 5) * 4 + (kblock & 3);
}

// Two fp32 to e4m3 (nearest even), lo in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// Eight fp32 to e2m1 (nearest even, larger ones to 6), first in the low nibble.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Value of an e2m1 code: its exponent and mantissa bits under the low exponent
// bits of fp32 read 2^-126 times the value (subnormals included).
__device__ __forceinline__ float e2m1_value(uint32_t code) {
  const float mag = __uint_as_float((code & 7u) << 22) * 0x1p126f;
  return (code & 8u) ? -mag : mag;
}

// A block of 32 fp32 to e4m3 codes (8 words); returns the scale byte.
__device__ __forceinline__ uint32_t mx8_block(const float (&v)[32], uint32_t (&codes)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  const int x = mx_exponent<8, kMxTopE4m3>(m);
  const float inv = mx_inverse(x);
  const bool bad = m >= 0x7f800000u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    codes[i] = e4m3x2(v[4 * i] * inv, v[4 * i + 1] * inv) | e4m3x2(v[4 * i + 2] * inv, v[4 * i + 3] * inv) << 16;
    if (bad) codes[i] = 0x7f7f7f7fu;
  }
  return bad ? 255u : (uint32_t)(x + 127);
}

}  // namespace moe
