// Device side of the 4-bit microscaled values (layout at hinm_mx4_t).
#ifndef HINM_MX4_H_
#define HINM_MX4_H_

#include "hinm_device.h"

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 2^(e - 127) as fp32; 255 is NaN, and 0 (2^-127) is subnormal.
__device__ inline float mx4_scale(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7fc00000u : e << 23);
}

// Eight codes times their scale, as bf16 (exact).
__device__ inline bf16x8 mx4_expand(uint32_t c, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return __builtin_shufflevector(__builtin_shufflevector(a, b, 0, 1, 2, 3), __builtin_shufflevector(d, e, 0, 1, 2, 3),
                                 0, 1, 2, 3, 4, 5, 6, 7);
}

}  // namespace

#endif  // HINM_MX4_H_
