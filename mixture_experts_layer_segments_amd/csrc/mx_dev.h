// MXFP4 on the device (OCP Microscaling formats, element type E2M1: sign,
// 2 exponent bits, 1 mantissa bit; values 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives).  32 consecutive elements of a row share one E8M0 scale, a byte b
// that stands for 2^(b - 127) (255: NaN); element 2i of a row sits in the low
// half of byte i.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace mx_dev {

// The scale as the conversion and matrix instructions take it in a float:
// its exponent field.
__device__ __forceinline__ float e8m0_float(uint32_t b) { return __uint_as_float(b << 23); }

// E8M0 byte of a block whose largest magnitude has the fp32 bits `abits`
// (sign cleared): the smallest s in [-127, 127] with amax <= 6 * 2^s, 0 for
// an all-zero block; 255 where a member is an infinity or NaN (their bit
// patterns are the largest).  amax = (1 + m / 2^23) * 2^E and 6 = 1.5 * 2^2,
// so s = E - 2 when the mantissa is at most 1.5 (m <= 0x400000), else E - 1.
// A subnormal amax is below 2^-126 and 6 * 2^-127 is not: s = -127.
__device__ __forceinline__ uint32_t block_e8m0(uint32_t abits) {
  if (abits == 0) return 127;
  if (abits >= 0x7f800000u) return 255;
  const int b = (int)(abits >> 23) - 2 + ((abits & 0x7fffffu) > 0x400000u ? 1 : 0);
  return (uint32_t)max(0, b);
}

// E2M1 codes of v[0..7] / 2^(b - 127), four bits each, v[0] lowest: the
// hardware conversion, to the nearest value, ties to even, sign kept.  (For
// a block with the NaN scale the codes are zeros.)
__device__ __forceinline__ uint32_t e2m1x8(const float* v, uint32_t b) {
  if (b == 255) return 0;
  const float sc = e8m0_float(b);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
  return w;
}

typedef uint32_t mx_u32x4 __attribute__((ext_vector_type(4)));

// The 8 codes of w times their block's scale, as 8 bf16 (exact: a bf16 holds
// every E2M1 value times every power of two of the format below overflow).
__device__ __forceinline__ mx_u32x4 e2m1x8_to_bf16(uint32_t w, float sc) {
  return mx_u32x4{
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, sc, 3))};
}

}  // namespace mx_dev
}  // namespace moe
