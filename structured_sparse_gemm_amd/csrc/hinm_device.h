// Device helpers shared by the product kernels of libhinm (not installed).
#ifndef HINM_DEVICE_H_
#define HINM_DEVICE_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ inline uint16_t bf16_rne(float f) {
  uint32_t u = __float_as_uint(f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return (uint16_t)((u >> 16) | 0x40u);  // NaN stays NaN
  u += 0x7fffu + ((u >> 16) & 1u);
  return (uint16_t)(u >> 16);
}

// Split-K hand-over: one workgroup of `splits` counts itself in on an
// agent-scope counter; true for the last to arrive.  The increment wraps (the
// hardware's atomic inc: old >= splits - 1 stores 0), so the counter is back
// at 0 after the last arrival without a separate store.
//
// Why the partial sums are visible to the last arriver without a cache
// writeback (gfx950 follows the gfx942 memory model of the LLVM AMDGPU
// back end): the partials are written and read only with agent-scope atomic
// stores and loads, which are issued with the sc1 bit and so are coherent
// across the XCDs' L2 caches (a store writes through to the device-coherent
// level, a load reads from it).  Each workgroup waits for its partial stores
// to be acknowledged (s_waitcnt vmcnt(0)) before its increment, and the last
// arriver issues its partial loads only after its increment has returned.
// A release / acquire pair would add an L2 writeback and invalidate, which
// are needed only for data written with ordinary stores; none is read here.
__device__ inline bool arrive(unsigned* ctr, int splits) {
  return __builtin_amdgcn_atomic_inc32(ctr, (unsigned)(splits - 1), __ATOMIC_RELAXED, "agent") ==
         (unsigned)(splits - 1);
}

// ds_read_b64_tr_b16: within each 16-lane group, output lane j receives
// element j%4 of the 8-byte segment addressed by lane 4q + j/4, for q = 0..3.
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ inline v4i16 tr_read(const uint16_t* lds_elem) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (lds_v4i16*)((__attribute__((address_space(3))) char*)((__attribute__((address_space(3))) uint16_t*)lds_elem)));
}

// Buffer resources (raw buffers, 32-bit offsets; an offset past the end
// reads zero).
constexpr int kBufferWord3 = 0x00020000;   // raw buffer, 32-bit data format (gfx9)
constexpr uint32_t kOob = 0xFFFFFFF0u;     // offset past every buffer: loads return zeros


typedef __attribute__((address_space(3))) uint8_t lds_u8;

// s_waitcnt with only the vector-memory count: vmcnt(n), nothing else.
template <int N>
__device__ inline void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}

// A buffer load whose 16 bytes per lane go straight to LDS: lane l's bytes
// land at lds + 16 l (an offset past the buffer writes zeros).  The sc0 bit
// (cache policy 1) makes the load miss in the CU's L1 and read from L2: a
// gathered X row is used once per workgroup, so L1 allocation buys nothing
// (0.5-1% faster on every batch-1024/2048 shape measured).
__device__ inline void load_lds16(__amdgpu_buffer_rsrc_t r, void* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)(lds_u8*)lds, 16, off, 0, 0, 1);
}

__device__ inline v4i16 tr_read_b(const uint8_t* lds) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(lds_u8*)lds);
}

}  // namespace

#endif  // HINM_DEVICE_H_
