// Blocks of 32 values in 4 bits that share a power of two (gfx950's conversions).
#ifndef KDA_CACHE4_H_
#define KDA_CACHE4_H_

#include "gfx950.h"

namespace kda {
namespace dev {

// The conversions read a scale's exponent field alone (whatever its sign and mantissa bits
// hold): a scale byte shifted to bits 23..30, with its neighbours still around it, is a scale.
// Field 255 gives NaN, as the byte 255 should.
__device__ __forceinline__ float scale_of(unsigned w, int byte) {
  return __uint_as_float(byte < 3 ? w << (23 - 8 * byte) : w >> 1);
}

// Byte SEL of w, two codes, to two bf16 times the scale (exact).
template <int SEL>
__device__ __forceinline__ unsigned two_values(unsigned w, float scale) {
  return __builtin_bit_cast(unsigned, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, SEL));
}
// Eight codes to eight bf16.
__device__ __forceinline__ u32x4_t eight_values(unsigned w, float scale) {
  return u32x4_t{two_values<0>(w, scale), two_values<1>(w, scale), two_values<2>(w, scale),
                 two_values<3>(w, scale)};
}

// The scale byte of a block whose largest magnitude has these bf16 bits (sign cleared): the
// smallest power of two that brings it within 6 = 1.5 2^2, so its own exponent less 2, or less
// 1 when its significand is above 1.5; 255 for infinities and NaN.
__device__ __forceinline__ unsigned scale_byte(unsigned top) {
  if (top >= 0x7f80u) return 255u;
  const int e = (int)((top + 0x3fu) >> 7) - 2;
  return (unsigned)max(e, 0);
}

// Eight bf16 to eight codes: nearest, ties to even (exact: a power of two divides).
__device__ __forceinline__ unsigned eight_codes(u32x4_t x, unsigned byte) {
  if (byte == 255u) return 0u;
  // a byte of zero is 2^-127, whose exponent field is zero as well
  const float s = __uint_as_float(byte << 23);
  unsigned w = 0u;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, bf_lo(x[0]), bf_hi(x[0]), s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, bf_lo(x[1]), bf_hi(x[1]), s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, bf_lo(x[2]), bf_hi(x[2]), s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, bf_lo(x[3]), bf_hi(x[3]), s, 3);
  return w;
}

}  // namespace dev
}  // namespace kda

#endif  // KDA_CACHE4_H_
