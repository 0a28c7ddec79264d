// 4-bit microscaled values of a packed weight (hinm_mx4_t): quantisation of
// the bf16 packed values and its inverse.  Both are one pass bound by memory
// traffic (2 bytes of bf16 and 17/32 bytes of 4-bit values a value).
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
};

// The scale byte of a block whose largest magnitude has the bf16 bits `top`.
__device__ inline int scale_of(uint32_t top) {
  const int field = (int)(top >> 7);                 // exponent field; 255: NaN or infinity
  return field == 255 ? 255 : max(field - 2, 0);
}

// E2M1 code of v / 2^(scale - 127): nearest, half-way cases to the even code.
__device__ inline uint32_t code_of(uint32_t bits, float inv) {
  const float a = fabsf(__uint_as_float(bits << 16)) * inv;    // exact: a power of two
  const uint32_t c = (a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) + (a > 5.f);
  return c | ((bits >> 12) & 8u);
}

// A workgroup per unit: thread 4r + q holds values 8q .. 8q+7 of row r, the
// four threads of a row agree on its largest magnitude, and the codes pass
// through LDS so that the stores are whole lines.
__global__ __launch_bounds__(256) void quantize_kernel(Mx4Region d, Mx4Region s) {
  __shared__ __attribute__((aligned(16))) uint32_t code[256];
  __shared__ __attribute__((aligned(16))) uint8_t scale[64];
  __shared__ __attribute__((aligned(16))) uint16_t meta[256];
  const int t = threadIdx.x, row = t >> 2, q = t & 3;
  for (int64_t w = blockIdx.x; w < d.units + s.units; w += gridDim.x) {
    const bool dense = w < d.units;
    const Mx4Region& r = dense ? d : s;
    const int64_t u = dense ? w : w - d.units;
    const u32x4 v = *reinterpret_cast<const u32x4*>(r.val + u * 2048 + 8 * t);
    uint32_t top = 0;
    for (int k = 0; k < 4; ++k) top = max(top, max(v[k] & 0x7fffu, (v[k] >> 16) & 0x7fffu));
    top = max(top, (uint32_t)__shfl_xor((int)top, 1));
    top = max(top, (uint32_t)__shfl_xor((int)top, 2));
    const int e = scale_of(top);
    const float inv = __uint_as_float((uint32_t)min(254 - e, 254) << 23);   // 2^(127 - e), e <= 252
    uint32_t c = 0;
    if (e != 255)
      for (int k = 0; k < 4; ++k)
        c |= (code_of(v[k] & 0xffffu, inv) << (8 * k)) | (code_of(v[k] >> 16, inv) << (8 * k + 4));
    const int at = (row & 15) * 4 + (row >> 4);
    code[q * 64 + at] = c;
    if (q == 0) scale[at] = (uint8_t)e;
    if (!dense) meta[q * 64 + at] = (uint16_t)(r.meta[u * 64 + row] >> (16 * q));
    __syncthreads();
    r.code[u * 256 + t] = code[t];
    if (t < 16) reinterpret_cast<uint32_t*>(r.scale + u * 64)[t] = reinterpret_cast<const uint32_t*>(scale)[t];
    if (!dense && t < 128)
      reinterpret_cast<uint32_t*>(r.meta4 + u * 256)[t] = reinterpret_cast<const uint32_t*>(meta)[t];
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void dequantize_kernel(Mx4Region d, Mx4Region s) {
  __shared__ __attribute__((aligned(16))) uint32_t code[256];
  __shared__ __attribute__((aligned(16))) uint8_t scale[64];
  __shared__ __attribute__((aligned(16))) uint16_t meta[256];
  const int t = threadIdx.x, row = t >> 2, q = t & 3;
  for (int64_t w = blockIdx.x; w < d.units + s.units; w += gridDim.x) {
    const bool dense = w < d.units;
    const Mx4Region& r = dense ? d : s;
    const int64_t u = dense ? w : w - d.units;
    code[t] = r.code[u * 256 + t];
    if (t < 16) reinterpret_cast<uint32_t*>(scale)[t] = reinterpret_cast<const uint32_t*>(r.scale + u * 64)[t];
    if (!dense && t < 128)
      reinterpret_cast<uint32_t*>(meta)[t] = reinterpret_cast<const uint32_t*>(r.meta4 + u * 256)[t];
    __syncthreads();
    const int at = (row & 15) * 4 + (row >> 4);
    *reinterpret_cast<u32x4*>(r.val + u * 2048 + 8 * t) =
        __builtin_bit_cast(u32x4, mx4_expand(code[q * 64 + at], mx4_scale(scale[at])));
    if (!dense && q == 0)
      r.meta[u * 64 + row] = (uint64_t)meta[at] | ((uint64_t)meta[64 + at] << 16) | ((uint64_t)meta[128 + at] << 32) |
                             ((uint64_t)meta[192 + at] << 48);
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void copy_words_kernel(const u32x4* __restrict__ a, u32x4* __restrict__ b, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) b[i] = a[i];
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

int copy_lists(const int32_t* a, int32_t* b, int64_t bytes, hipStream_t stream) {
  if (bytes == 0 || a == b) return HINM_OK;
  const int64_t n = bytes / 16;
  hipLaunchKernelGGL(copy_words_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 2048)), dim3(256), 0, stream,
                     reinterpret_cast<const u32x4*>(a), reinterpret_cast<u32x4*>(b), n);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? HINM_OK : fail(HINM_EHIP, "mx4 launch: %s", hipGetErrorString(e));
}

int convert(const hinm_plan_t& p, int32_t n, const hinm_packed_t& full, const hinm_mx4_t& four, bool quantize,
            void* stream_) {
  if (p.tile_rows % 64 != 0) return fail(HINM_ESHAPE, "tile_rows=%d is not a multiple of 64", p.tile_rows);
  if (n < 1) return fail(HINM_EINVAL, "n_weights=%d must be positive", n);
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
  Mx4Region d{static_cast<uint16_t*>(full.val_dense), nullptr, four.val_dense, four.scale_dense, nullptr,
              (int64_t)n * (p.bytes_val_dense / 4096)};
  Mx4Region s{static_cast<uint16_t*>(full.val_24), full.meta_24, four.val_24, four.scale_24, four.meta_24,
              (int64_t)n * (p.bytes_val_24 / 4096)};
  const int64_t units = d.units + s.units;
  if (units > 0) {
    const dim3 grid((unsigned)std::min<int64_t>(units, 1 << 20));
    if (quantize) hipLaunchKernelGGL(quantize_kernel, grid, dim3(256), 0, stream, d, s);
    else hipLaunchKernelGGL(dequantize_kernel, grid, dim3(256), 0, stream, d, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(HINM_EHIP, "mx4 launch: %s", hipGetErrorString(e));
  }
  const int32_t *id = quantize ? full.idx_dense : four.idx_dense, *is = quantize ? full.idx_24 : four.idx_24;
  int32_t *od = quantize ? four.idx_dense : full.idx_dense, *os = quantize ? four.idx_24 : full.idx_24;
  st = copy_lists(id, od, n * p.bytes_idx_dense, stream);
  return st ? st : copy_lists(is, os, n * p.bytes_idx_24, stream);
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
