// Device helpers of the 8-bit cache: e4m3 codes, and the byte b of a row that stands for the
// power of two 2^(b - 127) its codes are multiplied by.
#pragma once

#include "serving_common.h"

namespace sfn {

// The bytes in use. Up to 2^119 every e4m3 multiple is finite in bf16 and fp32; from 2^-117 on
// every one is a normal number there.
constexpr int kExpLeast = 10, kExpMost = 246;

// The smallest byte whose power of two times 448 is not below `top`, a row's largest finite
// magnitude: of the significand only whether it is above 1.75 counts.
__device__ __forceinline__ int exp_of_row(float top) {
  return min(max((int)((__float_as_uint(top) + 0x1fffffu) >> 23) - 8, kExpLeast), kExpMost);
}

// 2^(b - 127), for any byte the nearest of those in use: cells that were never written hold anything.
__device__ __forceinline__ float scale_of(uint32_t b) {
  return __uint_as_float((uint32_t)min(max((int)b, kExpLeast), kExpMost) << 23);
}

// Four values as e4m3 (nearest, ties to even; NaN stays NaN), |v| <= 448.
__device__ __forceinline__ uint32_t pack_e4m3(float v0, float v1, float v2, float v3) {
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v2, v3, lo, true);
}

// Two codes' values times `scale` as bf16, exactly: the low two bytes of the word, or the high two.
template <bool HIGH>
__device__ __forceinline__ uint32_t pair_of(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, HIGH));
}

// e4m3's NaN is the codes 0x7f and 0xff; it has no infinities.
__device__ __forceinline__ bool not_a_number(uint32_t code) { return (code & 0x7fu) == 0x7fu; }
// The top bit of each byte of the word that is one of them.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// The word with those bytes 0.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) { return w & ~((nan_codes(w) >> 7) * 0xffu); }

// Four codes' values times `scale`.
__device__ __forceinline__ void values_of(uint32_t codes, float scale, float* f) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, scale, false);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes, scale, true);
  f[0] = a[0];
  f[1] = a[1];
  f[2] = b[0];
  f[3] = b[1];
}

}  // namespace sfn
