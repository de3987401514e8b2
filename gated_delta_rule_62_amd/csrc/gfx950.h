// Small device helpers of the serving operators' kernels (gfx950, 64-lane waves).
#ifndef KDA_GFX950_H_
#define KDA_GFX950_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {
namespace dev {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned u32x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf2f(u16 x) { return __uint_as_float((unsigned)x << 16); }
__device__ __forceinline__ float bf_lo(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(unsigned w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats -> two bf16 (round to nearest even), the first in the low half.
__device__ __forceinline__ unsigned pack_bf16(float lo, float hi) {
  f32x2_t f = {lo, hi};
  return __builtin_bit_cast(unsigned, __builtin_convertvector(f, bf16x2_t));
}

// The one matrix shape of this library: 16x16 fp32 += 16x32 bf16 times 32x16 bf16.
// Lane l holds eight consecutive reduction slots 8*(l/16) .. of row (A) or column (B)
// l%16, and rows 4*(l/16) .. +3 of column l%16 of the accumulator.
__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf,
                                                            0xf, false));
}

// v of this 16-lane row plus (or the larger of it and) v of its pair row, in both rows:
// swapping the odd rows of one copy with the even rows of another leaves the pair's two
// values in the two results.  The 32-lane form pairs the wave's halves.
struct Two {
  float a, b;
};
__device__ __forceinline__ Two swap16(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  return Two{__uint_as_float(r[0]), __uint_as_float(r[1])};
}
__device__ __forceinline__ Two swap32(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  return Two{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

// Sum over aligned groups of G lanes, in every lane of the group.
template <int G>
__device__ __forceinline__ float group_sum(float v) {
  static_assert(G == 4 || G == 8 || G == 16 || G == 32, "group size");
  v += dpp<0xB1>(v);                          // quad_perm: lane xor 1
  v += dpp<0x4E>(v);                          // quad_perm: lane xor 2
  if constexpr (G >= 8) v += dpp<0x141>(v);   // row_half_mirror
  if constexpr (G >= 16) v += dpp<0x140>(v);  // row_mirror
  if constexpr (G >= 32) {
    const Two t = swap16(v);
    v = t.a + t.b;
  }
  return v;
}

// Sum over the wave, in every lane: of the lanes that differ in bit 0 of their number, then in bit
// 1, up to bit 5.  Where the compiler fuses the first addition with the product that v is, the
// lanes' sums differ in their last bits, and the order is part of the result.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(dpp<0x1B>(v));  // quads reversed, then halves of a row mirrored: lane xor 4
  v += dpp<0x128>(v);             // row_ror:8: lane xor 8
  Two t = swap16(v);
  v = t.a + t.b;
  t = swap32(v);
  return t.a + t.b;
}
// The same with mirrored lanes for bits 2 and 3.
__device__ __forceinline__ float wave_sum_mirrored(float v) {
  const Two t = swap32(group_sum<32>(v));
  return t.a + t.b;
}
// Maximum over the wave, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  Two t = swap16(v);
  v = fmaxf(t.a, t.b);
  t = swap32(v);
  return fmaxf(t.a, t.b);
}

// The last of n items for which `before` holds; it holds for a first part of them and counts as
// holding for the first.  Whole waves call it: 64 lanes look at once, where a binary search would
// wait for memory each step.
template <class F>
__device__ __forceinline__ int find_last(int n, F before) {
  const int lane = threadIdx.x & 63;
  int lo = 0;
  while (n > 1) {
    const int stride = (n + 63) >> 6, at = lane * stride;
    const int k = max(1, (int)__popcll(__ballot(at < n && before(lo + at)))) - 1;
    lo += k * stride;
    n = min(stride, n - k * stride);
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// Raw buffer descriptor over [base, base + bytes): loads past the end return zero and
// stores past it are dropped.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// Workgroup barrier that orders LDS only: global loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Four 16-bit values of one column from four rows: inside each 16-lane group, lane i
// receives element i%4 of the 8-byte pieces that lanes i/4, 4 + i/4, 8 + i/4 and
// 12 + i/4 address.
__device__ __forceinline__ u32x2_t ds_read_tr(const u16* p) {
  return __builtin_bit_cast(
      u32x2_t,
      __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)(p)));
}

// acc + 0 * (both bf16 of w): NaN from the first that is not finite.
__device__ __forceinline__ float dot_zero(unsigned w, float acc) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), bf16x2_t{(__bf16)0.f, (__bf16)0.f}, acc,
                                         false);
}

// Infinities and NaN in v at tokens that a row does not see: a matrix product would make a NaN
// of them and their zero weight.  Where any is, products take odd_split's `finite` (zeros in
// their place), and one of `code` with ones for the visible tokens counts the +inf, -inf and
// NaN of 32 tokens in steps of 1, 2^8 and 2^16, exact in fp32; odd_value is what a count adds
// to the row.
struct OddSplit {
  unsigned finite, code;
};
__device__ __forceinline__ OddSplit odd_split(unsigned w) {
  auto code = [](unsigned h) {  // one half
    const unsigned kind = (h & 0x7fu) != 0u ? 0x4780u : (h & 0x8000u) != 0u ? 0x4380u : 0x3f80u;
    return (h & 0x7f80u) == 0x7f80u ? kind : 0u;
  };
  const unsigned lo = code(w & 0xffffu), hi = code(w >> 16);
  return OddSplit{(lo ? 0u : w & 0xffffu) | (hi ? 0u : w & 0xffff0000u), lo | hi << 16};
}
__device__ __forceinline__ float odd_value(float count) {
  const unsigned n = (unsigned)count;
  const float inf = __builtin_inff(), plus = n & 0xff00ffu ? inf : 0.f;
  return n & 0xffff00u ? plus - inf : plus;
}

}  // namespace dev
}  // namespace kda

#endif  // KDA_GFX950_H_
