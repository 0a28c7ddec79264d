// Probe of how precisely gfx950's E4M3 matrix instructions add products, the
// reason why 8-bit codes are widened to bf16 ahead of the product (test
// infrastructure, not part of libhinm).
//
// Thirty-two products a[k] b[k] are added by one 16x16x64 SMFMAC that keeps
// positions 0 and 1 of every group of four, every row and column alike: once
// with E4M3 operands, once with the same values as bf16.
//   E4M3: lane l = 16 kc + i holds row i's compressed values 8kc..8kc+7 and of
//         column i the positions 16kc..16kc+15.
//   bf16: as in smfmac_probe.hip, the positions 8kc..8kc+7 and 32+8kc..32+8kc+7.
#include <hip/hip_runtime.h>
#include <stdint.h>

typedef int i32x2_t __attribute__((ext_vector_type(2)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x16_t __attribute__((ext_vector_type(16)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// a, b: 32 codes each; d: one float a lane.
__global__ __launch_bounds__(64) void e4m3_kernel(const uint8_t* a, const uint8_t* b, float* d) {
  const int kc = threadIdx.x >> 4;
  uint32_t av[2] = {0, 0}, bv[4] = {0, 0, 0, 0};
  for (int e = 0; e < 8; ++e) av[e / 4] |= (uint32_t)a[8 * kc + e] << (8 * (e % 4));
  for (int e = 0; e < 16; ++e)
    if (e % 4 < 2) bv[e / 4] |= (uint32_t)b[8 * kc + 2 * (e / 4) + e % 4] << (8 * (e % 4));
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  acc = __builtin_amdgcn_smfmac_f32_16x16x64_fp8_fp8(i32x2_t{(int)av[0], (int)av[1]},
                                                     i32x4_t{(int)bv[0], (int)bv[1], (int)bv[2], (int)bv[3]}, acc, 0x4444, 0, 0);
  d[threadIdx.x] = acc[0];
}

// a, b: 32 bf16 values each.
__global__ __launch_bounds__(64) void bf16_kernel(const uint16_t* a, const uint16_t* b, float* d) {
  const int kc = threadIdx.x >> 4;
  bf16x8_t av;
  bf16x16_t bv;
  for (int e = 0; e < 8; ++e) av[e] = __builtin_bit_cast(__bf16, a[8 * kc + e]);
  for (int e = 0; e < 16; ++e) {
    const int p = (e < 8 ? 0 : 32) + 8 * kc + e % 8;
    bv[e] = __builtin_bit_cast(__bf16, p % 4 < 2 ? b[2 * (p / 4) + p % 4] : (uint16_t)0);
  }
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  acc = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av, bv, acc, 0x4444, 0, 0);
  d[threadIdx.x] = acc[0];
}

// Device buffers: 32 codes or bf16 values each, 64 floats.  Waits; returns the
// HIP error code (0 on success).
extern "C" int e4m3_sums_probe(int e4m3, const void* a, const void* b, void* d) {
  if (e4m3)
    hipLaunchKernelGGL(e4m3_kernel, dim3(1), dim3(64), 0, 0, (const uint8_t*)a, (const uint8_t*)b, (float*)d);
  else
    hipLaunchKernelGGL(bf16_kernel, dim3(1), dim3(64), 0, 0, (const uint16_t*)a, (const uint16_t*)b, (float*)d);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? (int)e : (int)hipDeviceSynchronize();
}
