// Device side of the 8-bit floating-point values (layout at hinm_fp8_t).
#ifndef HINM_FP8_H_
#define HINM_FP8_H_

#include "hinm_device.h"

namespace {

typedef uint32_t fp8_u32x2 __attribute__((ext_vector_type(2)));

// 2^(e - 127) for 1 <= e <= 254: every scale is of 3 .. 246.
__device__ inline float fp8_scale(uint32_t e) { return __uint_as_float(e << 23); }
__device__ inline float fp8_inverse(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// The scale byte of a block whose largest finite magnitude has the bf16 bits
// `top`: 448 is 1.75 * 2^8, so a mantissa above 1.75 (0x60 of 7 bits) takes
// the next power of two.
__device__ inline uint32_t fp8_scale_of(uint32_t top) {
  const int e = (int)(top >> 7) - 8 + ((top & 0x7fu) > 0x60u ? 1 : 0);
  return (uint32_t)min(max(e, 3), 246);
}

// Larger of two pairs of bf16 magnitudes, NaN and infinity counting as 0.
__device__ inline uint32_t fp8_max_finite(uint32_t m, uint32_t v) {
  const uint32_t lo = v & 0x7fffu, hi = (v >> 16) & 0x7fffu;
  const uint32_t ml = m & 0xffffu, mh = m >> 16;
  return max(ml, lo < 0x7f80u ? lo : 0u) | (max(mh, hi < 0x7f80u ? hi : 0u) << 16);
}

// Two bf16 values (one dword) as E4M3 codes of v * inverse, in the low or high
// half of `old`.  The product is exact, the conversion rounds to nearest even;
// the clamp saturates (only values past 448 * 2^119 reach it).
template <bool HIGH>
__device__ inline uint32_t fp8_codes(uint32_t old, uint32_t v, float inverse) {
  const float a = __uint_as_float(v << 16), b = __uint_as_float(v & 0xffff0000u);
  const float x = __builtin_fminf(__builtin_fmaxf(a * inverse, -448.f), 448.f);
  const float y = __builtin_fminf(__builtin_fmaxf(b * inverse, -448.f), 448.f);
  uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x, y, (int)old, HIGH);
  constexpr int at = HIGH ? 16 : 0;
  if ((v & 0x7f80u) == 0x7f80u) c = (c & ~(0xffu << at)) | (0x7fu << at);
  if ((v & 0x7f800000u) == 0x7f800000u) c = (c & ~(0xff00u << at)) | (0x7f00u << at);
  return c;
}

// Eight bf16 values of one block.
__device__ inline fp8_u32x2 fp8_codes8(u32x4 v, float inverse) {
  fp8_u32x2 c;
  c[0] = fp8_codes<true>(fp8_codes<false>(0u, v[0], inverse), v[1], inverse);
  c[1] = fp8_codes<true>(fp8_codes<false>(0u, v[2], inverse), v[3], inverse);
  return c;
}

// Eight codes times their scale, as bf16 (exact; the NaN code stays NaN).
__device__ inline u32x4 fp8_expand(fp8_u32x2 c, float scale) {
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], scale, false));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], scale, true));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], scale, false));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], scale, true));
  return v;
}

}  // namespace

#endif  // HINM_FP8_H_
