// 4-bit microscaled values of a packed weight (hinm_mx4_t): quantisation of
// the bf16 packed values and its inverse.  Both are one pass bound by memory
// traffic (2 bytes of bf16 and 17/32 bytes of 4-bit values a value): 8 weights
// of 11008x4096 take 49 us to quantise and 44 back, 4.0 and 4.5 TB/s with the index
// lists and metadata.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hinm_device.h"
#include "hinm_internal.h"
#include "hinm_mx4.h"

using hinm::fail;

namespace {

// One region (dense or 2:4) of all weights: `units` K-block x 64-row units of
// 4 KiB of bf16 values each.  Source rows lie [block][tile_rows][32], so unit
// u is the u-th 4 KiB; the 4-bit side keeps the same order of units.
struct Mx4Region {
  uint16_t* val;
  uint64_t* meta;          // 2:4 only
  uint32_t* code;
  uint8_t* scale;
  uint16_t* meta4;
  int64_t units;
  const u32x4* idx;        // index lists, copied as they are
  u32x4* idx_out;
  int64_t idx_words;       // of 16 bytes; 0: nothing to copy
};

// The workgroups' share of the list copies.
__device__ inline void copy_lists(const Mx4Region& r) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < r.idx_words; i += (int64_t)gridDim.x * 256)
    r.idx_out[i] = r.idx[i];
}

// The scale byte of a block whose largest magnitude has the bf16 bits `top`.
__device__ inline int scale_of(uint32_t top) {
  const int field = (int)(top >> 7);                 // exponent field; 255: NaN or infinity
  return field == 255 ? 255 : max(field - 2, 0);
}

// Eight bf16 values as E2M1 codes of v / scale: the conversion rounds half-way
// cases to the even code and saturates at 6.
__device__ inline uint32_t codes_of(u32x4 v, float scale) {
  const uint32_t w0 = v[0], w1 = v[1], w2 = v[2], w3 = v[3];
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w0), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w1), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w2), scale, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, w3), scale, 3);
  return c;
}

// The largest magnitude (as bf16 bits) of the 32 values that four adjacent
// lanes hold.
__device__ inline uint32_t top_of(u32x4 v) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 m = __builtin_bit_cast(u16x2, v[0] & 0x7fff7fffu);
#pragma unroll
  for (int c = 1; c < 4; ++c) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[c] & 0x7fff7fffu));
  uint32_t top = max(m[0], m[1]);
  top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xf, 0xf, true));   // lane ^ 1
  return max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xf, 0xf, true));  // lane ^ 2
}

// A workgroup takes kUnits units at a time, so that each thread has that many
// loads in flight between two barriers (one unit at a time: 81 us for 8
// weights of 11008x4096).  Thread 4r + q holds values 8q .. 8q+7 of row r, the
// four threads of a row agree on its largest magnitude, and the codes pass
// through LDS so that the stores are whole lines.
constexpr int kUnits = 4;

struct Staged {
  uint32_t code[256];
  uint32_t meta[128];      // uint16 [4][16][4]
  uint32_t scale[16];      // uint8 [16][4]
};

__global__ __launch_bounds__(256) void quantize_kernel(Mx4Region d, Mx4Region s) {
  __shared__ __attribute__((aligned(16))) Staged st[kUnits];
  const int t = threadIdx.x, row = t >> 2, q = t & 3, at = (row & 15) * 4 + (row >> 4);
  copy_lists(d);
  copy_lists(s);
  const int64_t all = d.units + s.units;
  for (int64_t w0 = (int64_t)blockIdx.x * kUnits; w0 < all; w0 += (int64_t)gridDim.x * kUnits) {
    u32x4 v[kUnits];
    uint64_t m[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int64_t w = min(w0 + k, all - 1);
      const bool dense = w < d.units;
      const int64_t u = dense ? w : w - d.units;
      v[k] = *reinterpret_cast<const u32x4*>((dense ? d.val : s.val) + u * 2048 + 8 * t);
      m[k] = dense ? 0ull : s.meta[u * 64 + row];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int e = scale_of(top_of(v[k]));
      const uint32_t code = e == 255 ? 0u : codes_of(v[k], mx4_scale((uint32_t)e));
      st[k].code[q * 64 + at] = code;
      reinterpret_cast<uint16_t*>(st[k].meta)[q * 64 + at] = (uint16_t)(m[k] >> (16 * q));
      if (q == 0) reinterpret_cast<uint8_t*>(st[k].scale)[at] = (uint8_t)e;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int64_t w = w0 + k;
      if (w >= all) break;
      const bool dense = w < d.units;
      const int64_t u = dense ? w : w - d.units;
      (dense ? d.code : s.code)[u * 256 + t] = st[k].code[t];
      if (t < 16) reinterpret_cast<uint32_t*>((dense ? d.scale : s.scale) + u * 64)[t] = st[k].scale[t];
      if (!dense && t < 128) reinterpret_cast<uint32_t*>(s.meta4 + u * 256)[t] = st[k].meta[t];
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void dequantize_kernel(Mx4Region d, Mx4Region s) {
  __shared__ __attribute__((aligned(16))) Staged st[kUnits];
  const int t = threadIdx.x, row = t >> 2, q = t & 3, at = (row & 15) * 4 + (row >> 4);
  copy_lists(d);
  copy_lists(s);
  const int64_t all = d.units + s.units;
  for (int64_t w0 = (int64_t)blockIdx.x * kUnits; w0 < all; w0 += (int64_t)gridDim.x * kUnits) {
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int64_t w = min(w0 + k, all - 1);
      const bool dense = w < d.units;
      const int64_t u = dense ? w : w - d.units;
      st[k].code[t] = (dense ? d.code : s.code)[u * 256 + t];
      if (t < 16) st[k].scale[t] = reinterpret_cast<const uint32_t*>((dense ? d.scale : s.scale) + u * 64)[t];
      if (!dense && t < 128) st[k].meta[t] = reinterpret_cast<const uint32_t*>(s.meta4 + u * 256)[t];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int64_t w = w0 + k;
      if (w >= all) break;
      const bool dense = w < d.units;
      const int64_t u = dense ? w : w - d.units;
      const float scale = mx4_scale(reinterpret_cast<const uint8_t*>(st[k].scale)[at]);
      // past the caches: 71 us without the hint for 8 weights of 11008x4096, 45 with it
      __builtin_nontemporal_store(__builtin_bit_cast(u32x4, mx4_expand(st[k].code[q * 64 + at], scale)),
                                  reinterpret_cast<u32x4*>((dense ? d.val : s.val) + u * 2048 + 8 * t));
      if (!dense && t < 64) {                    // row t: its four 16-bit pieces
        const uint16_t* m = reinterpret_cast<const uint16_t*>(st[k].meta) + (t & 15) * 4 + (t >> 4);
        s.meta[u * 64 + t] = (uint64_t)m[0] | ((uint64_t)m[64] << 16) | ((uint64_t)m[128] << 32) | ((uint64_t)m[192] << 48);
      }
    }
    __syncthreads();
  }
}

struct Buf {
  const void* ptr;
  int64_t bytes;
  const char* name;
};

int check_bufs(const Buf* b, int n, const char* whose) {
  for (int i = 0; i < n; ++i) {
    if (b[i].bytes > 0 && !b[i].ptr)
      return fail(HINM_EINVAL, "%s: %s is NULL but holds %lld bytes", whose, b[i].name, (long long)b[i].bytes);
    if (!hinm::aligned(b[i].ptr, 16)) return fail(HINM_EALIGN, "%s: %s is not 16-byte aligned", whose, b[i].name);
  }
  return HINM_OK;
}

int convert(const hinm_plan_t& p, int64_t n, const hinm_packed_t& full, const hinm_mx4_t& four, bool quantize,
            void* stream_) {
  if (p.tile_rows % 64 != 0) return fail(HINM_ESHAPE, "tile_rows=%d is not a multiple of 64", p.tile_rows);
  if (n < 1) return fail(HINM_EINVAL, "n_weights=%lld must be positive", (long long)n);
  const Buf fb[5] = {{full.val_dense, p.bytes_val_dense, "val_dense"}, {full.idx_dense, p.bytes_idx_dense, "idx_dense"},
                     {full.val_24, p.bytes_val_24, "val_24"}, {full.meta_24, p.bytes_meta_24, "meta_24"},
                     {full.idx_24, p.bytes_idx_24, "idx_24"}};
  const Buf qb[7] = {{four.val_dense, p.bytes_val_dense, "val_dense"}, {four.scale_dense, p.bytes_val_dense, "scale_dense"},
                     {four.idx_dense, p.bytes_idx_dense, "idx_dense"}, {four.val_24, p.bytes_val_24, "val_24"},
                     {four.scale_24, p.bytes_val_24, "scale_24"}, {four.meta_24, p.bytes_meta_24, "meta_24"},
                     {four.idx_24, p.bytes_idx_24, "idx_24"}};
  int st = check_bufs(fb, 5, "bf16 weight");
  if (st) return st;
  st = check_bufs(qb, 7, "4-bit weight");
  if (st) return st;
  st = hinm::ensure_device();
  if (st) return st;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  const int32_t *id = quantize ? full.idx_dense : four.idx_dense, *is = quantize ? full.idx_24 : four.idx_24;
  int32_t *od = quantize ? four.idx_dense : full.idx_dense, *os = quantize ? four.idx_24 : full.idx_24;
  const Mx4Region d{static_cast<uint16_t*>(full.val_dense), nullptr, four.val_dense, four.scale_dense, nullptr,
                    n * (p.bytes_val_dense / 4096), reinterpret_cast<const u32x4*>(id), reinterpret_cast<u32x4*>(od),
                    id == od ? 0 : n * (p.bytes_idx_dense / 16)};
  const Mx4Region s{static_cast<uint16_t*>(full.val_24), full.meta_24, four.val_24, four.scale_24, four.meta_24,
                    n * (p.bytes_val_24 / 4096), reinterpret_cast<const u32x4*>(is), reinterpret_cast<u32x4*>(os),
                    is == os ? 0 : n * (p.bytes_idx_24 / 16)};
  const int64_t units = d.units + s.units;
  if (units > 0) {
    const dim3 grid((unsigned)std::min<int64_t>((units + kUnits - 1) / kUnits, 1 << 20));
    if (quantize) hipLaunchKernelGGL(quantize_kernel, grid, dim3(256), 0, stream, d, s);
    else hipLaunchKernelGGL(dequantize_kernel, grid, dim3(256), 0, stream, d, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(HINM_EHIP, "mx4 launch: %s", hipGetErrorString(e));
  }
  return HINM_OK;
}

}  // namespace

extern "C" int hinm_mx4_quantize(const hinm_packed_t* packed, int32_t n_weights, hinm_mx4_t* out, void* stream) {
  hinm::clear_error();
  if (!packed || !out) return fail(HINM_EINVAL, "packed and out must be non-NULL");
  int st = hinm::check_plan(&packed->plan);
  if (st) return st;
  st = convert(packed->plan, n_weights, *packed, *out, true, stream);
  if (st == HINM_OK) out->plan = packed->plan;
  return st;
}

extern "C" int hinm_mx4_dequantize(const hinm_mx4_t* packed, int32_t n_weights, hinm_packed_t* out, void* stream) {
  hinm::clear_error();
  if (!packed || !out) return fail(HINM_EINVAL, "packed and out must be non-NULL");
  int st = hinm::check_plan(&packed->plan);
  if (st) return st;
  st = convert(packed->plan, n_weights, *out, *packed, false, stream);
  if (st == HINM_OK) {
    out->plan = packed->plan;
    out->flags = 0;
    out->reserved = 0;
  }
  return st;
}
