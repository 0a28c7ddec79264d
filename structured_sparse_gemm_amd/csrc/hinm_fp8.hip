// 8-bit floating-point values of a packed weight (hinm_fp8_t): quantisation of
// the bf16 packed values and its inverse.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hinm_device.h"
#include "hinm_fp8.h"
#include "hinm_internal.h"

using hinm::Buf;
using hinm::check_bufs;
using hinm::fail;

namespace {

// One region (dense or 2:4) of all weights.  A unit is 64 rows of four
// K-blocks that share a scale (the region's last group may have fewer).
struct Fp8Region {
  uint16_t* val;
  uint8_t* code;
  uint8_t* scale;
  int nkb, ngr, rows;      // K-blocks and groups of a tile, tile height
  int64_t units;           // n_weights * n_tiles * ngr * rows / 64
  const u32x4 *idx, *meta; // lists and metadata, copied as they are
  u32x4 *idx_out, *meta_out;
  int64_t idx_words, meta_words;   // of 16 bytes; 0: nothing to copy
};

__device__ inline void copy_lists(const Fp8Region& r) {
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  for (int64_t i = i0; i < r.idx_words; i += step) r.idx_out[i] = r.idx[i];
  for (int64_t i = i0; i < r.meta_words; i += step) r.meta_out[i] = r.meta[i];
}

// Where unit u lies: its first K-block's value offset (elements), the blocks
// it holds and its scale bytes.
struct Fp8Unit {
  int64_t val, scale, stride;
  int blocks;
};
__device__ inline Fp8Unit unit_of(const Fp8Region& r, int64_t u) {
  const int chunks = r.rows / 64;
  const int c = (int)(u % chunks);
  const int64_t tg = u / chunks;
  const int g = (int)(tg % r.ngr);
  const int64_t t = tg / r.ngr;
  return {((t * r.nkb + 4 * g) * r.rows + 64 * c) * 32, tg * r.rows + 64 * c, (int64_t)r.rows * 32, min(4, r.nkb - 4 * g)};
}

// Thread 4 row + q holds values 8 q .. 8 q + 7 of the row in each of the four
// blocks: four 16-byte loads in flight, stores of 512 bytes a wave.
__global__ __launch_bounds__(256) void fp8_quantize_kernel(Fp8Region d, Fp8Region s) {
  copy_lists(d);
  copy_lists(s);
  const int64_t all = d.units + s.units;
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    const bool dense = w < d.units;
    const Fp8Region& r = dense ? d : s;
    const Fp8Unit u = unit_of(r, dense ? w : w - d.units);
    u32x4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = k < u.blocks ? *reinterpret_cast<const u32x4*>(r.val + u.val + k * u.stride + 8 * threadIdx.x)
                          : u32x4{0u, 0u, 0u, 0u};
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int c = 0; c < 4; ++c) m = fp8_max_finite(m, v[k][c]);
    uint32_t top = max(m & 0xffffu, m >> 16);
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xf, 0xf, true));   // lane ^ 1
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xf, 0xf, true));   // lane ^ 2
    const uint32_t e = fp8_scale_of(top);
    const float inverse = fp8_inverse(e);
    if ((threadIdx.x & 3) == 0) r.scale[u.scale + (threadIdx.x >> 2)] = (uint8_t)e;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < u.blocks)
        *reinterpret_cast<fp8_u32x2*>(r.code + u.val + k * u.stride + 8 * threadIdx.x) = fp8_codes8(v[k], inverse);
  }
}

__global__ __launch_bounds__(256) void fp8_dequantize_kernel(Fp8Region d, Fp8Region s) {
  copy_lists(d);
  copy_lists(s);
  const int64_t all = d.units + s.units;
  for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
    const bool dense = w < d.units;
    const Fp8Region& r = dense ? d : s;
    const Fp8Unit u = unit_of(r, dense ? w : w - d.units);
    fp8_u32x2 c[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = k < u.blocks ? *reinterpret_cast<const fp8_u32x2*>(r.code + u.val + k * u.stride + 8 * threadIdx.x)
                          : fp8_u32x2{0u, 0u};
    const float scale = fp8_scale(r.scale[u.scale + (threadIdx.x >> 2)]);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < u.blocks)
        *reinterpret_cast<u32x4*>(r.val + u.val + k * u.stride + 8 * threadIdx.x) = fp8_expand(c[k], scale);
  }
}

int convert(const hinm_plan_t& p, int64_t n, const hinm_packed_t& full, const hinm_fp8_t& eight, bool quantize,
            void* stream_) {
  if (p.tile_rows % 64 != 0) return fail(HINM_ESHAPE, "tile_rows=%d is not a multiple of 64", p.tile_rows);
  if (n < 1) return fail(HINM_EINVAL, "n_weights=%lld must be positive", (long long)n);
  const Buf fb[5] = {{full.val_dense, p.bytes_val_dense, "val_dense"}, {full.idx_dense, p.bytes_idx_dense, "idx_dense"},
                     {full.val_24, p.bytes_val_24, "val_24"}, {full.meta_24, p.bytes_meta_24, "meta_24"},
                     {full.idx_24, p.bytes_idx_24, "idx_24"}};
  const Buf qb[7] = {{eight.val_dense, p.bytes_val_dense, "val_dense"}, {eight.scale_dense, p.bytes_val_dense, "scale_dense"},
                     {eight.idx_dense, p.bytes_idx_dense, "idx_dense"}, {eight.val_24, p.bytes_val_24, "val_24"},
                     {eight.scale_24, p.bytes_val_24, "scale_24"}, {eight.meta_24, p.bytes_meta_24, "meta_24"},
                     {eight.idx_24, p.bytes_idx_24, "idx_24"}};
  int st = check_bufs(fb, 5, "bf16 weight");
  if (st) return st;
  st = check_bufs(qb, 7, "8-bit weight");
  if (st) return st;
  st = hinm::ensure_device();
  if (st) return st;
  const bool q = quantize;
  const int32_t *id = q ? full.idx_dense : eight.idx_dense, *is = q ? full.idx_24 : eight.idx_24;
  int32_t *od = q ? eight.idx_dense : full.idx_dense, *os = q ? eight.idx_24 : full.idx_24;
  const uint64_t* im = q ? full.meta_24 : eight.meta_24;
  uint64_t* om = q ? eight.meta_24 : full.meta_24;
  const int64_t chunks = n * p.n_tiles * (p.tile_rows / 64);
  const int kd = p.n_dense_pad / HINM_KB_DENSE, ks = p.n_24_pad / HINM_KB_24;
  const Fp8Region d{static_cast<uint16_t*>(full.val_dense), eight.val_dense, eight.scale_dense, kd, (kd + 3) / 4,
                    p.tile_rows, chunks * ((kd + 3) / 4), reinterpret_cast<const u32x4*>(id), nullptr,
                    reinterpret_cast<u32x4*>(od), nullptr, id == od ? 0 : n * (p.bytes_idx_dense / 16), 0};
  const Fp8Region s{static_cast<uint16_t*>(full.val_24), eight.val_24, eight.scale_24, ks, (ks + 3) / 4,
                    p.tile_rows, chunks * ((ks + 3) / 4), reinterpret_cast<const u32x4*>(is),
                    reinterpret_cast<const u32x4*>(im), reinterpret_cast<u32x4*>(os), reinterpret_cast<u32x4*>(om),
                    is == os ? 0 : n * (p.bytes_idx_24 / 16), im == om ? 0 : n * (p.bytes_meta_24 / 16)};
  const int64_t units = d.units + s.units;
  if (units > 0) {
    const dim3 grid((unsigned)std::min<int64_t>(units, 1 << 20));
    hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
    if (q) hipLaunchKernelGGL(fp8_quantize_kernel, grid, dim3(256), 0, stream, d, s);
    else hipLaunchKernelGGL(fp8_dequantize_kernel, grid, dim3(256), 0, stream, d, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(HINM_EHIP, "8-bit values' launch: %s", hipGetErrorString(e));
  }
  return HINM_OK;
}

}  // namespace

extern "C" int hinm_fp8_quantize(const hinm_packed_t* packed, int32_t n_weights, hinm_fp8_t* out, void* stream) {
  hinm::clear_error();
  if (!packed || !out) return fail(HINM_EINVAL, "packed and out must be non-NULL");
  int st = hinm::check_plan(&packed->plan);
  if (st) return st;
  st = convert(packed->plan, n_weights, *packed, *out, true, stream);
  if (st == HINM_OK) out->plan = packed->plan;
  return st;
}

extern "C" int hinm_fp8_dequantize(const hinm_fp8_t* packed, int32_t n_weights, hinm_packed_t* out, void* stream) {
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
