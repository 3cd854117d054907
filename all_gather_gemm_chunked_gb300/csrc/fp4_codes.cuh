// fp4_codes.cuh -- microscaled e2m1: the scale of a block of 32 elements and the codes.
//
// The scale is 2^E, E from the exponent of the block's largest magnitude m = f * 2^e (f
// from 1 on, below 2): E = e - 2, so that m / 2^E lies from 4 on, and e - 1 where f >=
// 1.75: 7 and above would round to 8, which is no code (the largest is 6), and below 7 a
// code is off by at most half its step.  In bits: adding 2^21 to the float carries into the
// exponent from 1.75 on.  Dividing by a power of two is exact, so a code is the nearest to
// the element itself.

#pragma once

#include <stdint.h>

namespace agg {

constexpr int kMicroBlock = 32;

// The magnitude's bits: they order as the magnitudes do, an infinity behind every number
// and NaN behind that.
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The scale's byte, E + 127, of a block whose largest magnitude has these bits; 255 (NaN)
// where it is not finite.
__device__ __forceinline__ uint32_t micro_scale(uint32_t largest) {
  const int32_t e = static_cast<int32_t>((largest + 0x200000u) >> 23) - 2;
  return largest >= 0x7f800000u ? 255u : static_cast<uint32_t>(e > 0 ? e : 0);
}
// 2^-E: 2^127 for byte 0, 2^-126 for 253, the largest of a finite block.
__device__ __forceinline__ float micro_inverse(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight codes, the first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

}  // namespace agg
