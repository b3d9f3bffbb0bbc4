// e4m3 values with power-of-two scales: the scale of a group is the smallest
// 2^e with max|x| <= 448 * 2^e, e kept within -120..120 (-120 for zeros),
// stored as e8m0 (e + 127).
#pragma once

#include "common.h"

namespace bd {

// e + 127 for a group whose largest magnitude is amax.  448 = 1.75 * 2^8, so
// with amax = 1.m * 2^E the exponent is E - 8, one more where 1.m > 1.75.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)min(max(e, 7), 247);
}

// 2^-(e) of a scale byte e + 127 (7..247: both signs of e are normal floats).
__device__ __forceinline__ float inv_scale(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// The value that a cached group's magnitudes are held to: the largest e4m3
// value below 2^128 at the largest scale is 240 * 2^120.
__device__ __forceinline__ float hold_e4m3(float x) {
  const float top = __uint_as_float(0x7F700000u);  // 1.875 * 2^127
  return x > top ? top : (x < -top ? -top : x);    // a NaN stays
}

// Four floats, already divided by their scale, to e4m3 (nearest even).
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

// Two e4m3 bytes (the low or the high half of v) times a power of two, as
// packed bf16: exact wherever the result is a bf16 number.
template <bool HI>
__device__ __forceinline__ uint32_t bf16x2_of_e4m3(uint32_t v, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, scale, HI));
}

}  // namespace bd
