// e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives; two a byte, the
// even one low) with one power-of-two scale for 32 of them: the smallest 2^e
// with max|x| <= 6 * 2^e, e kept within -120..120 (-120 for zeros), stored as
// e8m0 (e + 127).  e2m1 has no NaN: a group that holds one gets e8m0's, 255,
// and is NaN as a whole.
#pragma once

#include "common.h"

namespace bd {

constexpr int kGroup4 = 32;        // dims of a row that share a scale
constexpr uint32_t kNanScale = 255;

// The value that a group's magnitudes are held to: 6 at the largest scale.
__device__ __forceinline__ float hold_e2m1(float x) {
  const float top = __uint_as_float(0x7CC00000u);  // 1.5 * 2^122
  return x > top ? top : (x < -top ? -top : x);    // a NaN stays
}

// The scale byte of a group by the bits of its largest magnitude; those of a
// NaN are larger than a number's.  6 = 1.5 * 2^2, so with 1.m * 2^E the
// exponent is E - 2, one more where 1.m > 1.5.
__device__ __forceinline__ uint32_t scale_byte4(uint32_t bits) {
  const int e = (int)(bits >> 23) - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return bits > 0x7F800000u ? kNanScale : (uint32_t)min(max(e, 7), 247);
}

// Eight floats over a power of two to e2m1, nearest with ties to the even code.
__device__ __forceinline__ uint32_t pack_e2m1(const float (&f)[8], float scale) {
  uint32_t r = 0u;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[0], f[1], scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[2], f[3], scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[4], f[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, f[6], f[7], scale, 3);
}

// Eight e2m1 values times a power of two as packed bf16: exact wherever the
// result is a bf16 number.  The conversion takes the scale's exponent bits
// alone, which are the e8m0 byte: 0 counts as 2^-127 and 255 gives NaN.
__device__ __forceinline__ u32x4 bf16x8_of_e2m1(uint32_t v, float scale) {
  return u32x4{
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v, scale, 3))};
}

}  // namespace bd
