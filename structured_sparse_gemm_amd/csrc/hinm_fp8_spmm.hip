// hinm_spmm_fp8, hinm_spmm_experts_fp8: products of packed weights with 8-bit
// values and activations rounded to 8 bits token by token (layout and formulas
// at hinm_fp8_t).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hinm_device.h"
#include "hinm_fp8.h"
#include "hinm_internal.h"
#include "hinm_ragged.h"

using hinm::fail;

namespace {

// ds_read_b64_tr_b8: within each 16-lane group, lane 2 p + s addresses eight
// bytes (tokens 8 s .. 8 s + 7) of position p; output lane j receives token
// j's bytes of positions 0 .. 7.
__device__ inline fp8_u32x2 tr_read8(const uint8_t* lds) {
  typedef int v2i32 __attribute__((ext_vector_type(2)));
  typedef __attribute__((address_space(3))) v2i32 lds_v2i32;
  return __builtin_bit_cast(fp8_u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i32*)(lds_u8*)lds));
}

// The weights of all experts, the activations and a window of their columns.
// Strides are per expert.
struct Fp8Args {
  const uint8_t *val_d, *val_s, *scale_d, *scale_s;
  const uint64_t* meta;
  const int32_t *idx_d, *idx_s;
  int64_t n_val_d, n_val_s, n_scale_d, n_scale_s, n_meta, n_idx_d, n_idx_s;   // elements of one expert
  const uint16_t* x;                 // bf16 [cin][ldx]
  int64_t ldx;
  const uint8_t* x8;                 // E4M3 [cin][ld8], columns col0 .. col1 - 1; E8M0 xs [ld8]
  const uint8_t* xs;
  int ld8, col0, col1;
  uint16_t* y;
  int64_t ldy;
  const int32_t *starts, *counts;    // NULL: one range, all columns
  int n_experts, n_cols;
  int cin, cout, rows, n_tiles, nkb_d, nkb_s;
};

// ---------------------------------------------------------------------------
// Activations to 8 bits.  The scale of a token needs its whole column, so one
// kernel takes the largest magnitudes of kChunks pieces of the channels and a
// second one combines them and rounds; the second read of X comes from the
// last-level cache.
// ---------------------------------------------------------------------------
constexpr int kChunks = 64;          // pieces of the channels

// Eight columns of a row, zeros past the last one.
__device__ inline u32x4 load_row8(const uint16_t* row, int n, int n_cols) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (n + 8 <= n_cols) return *reinterpret_cast<const any_u32x4*>(row + n);
  for (int u = 0; u < 8 && n + u < n_cols; ++u) v[u >> 1] |= (uint32_t)row[n + u] << (16 * (u & 1));
  return v;
}

// Workgroup: 256 columns (32 threads of 8), 8 rows at a time of one piece.
__global__ __launch_bounds__(256) void fp8_colmax_kernel(Fp8Args a, uint16_t* __restrict__ part) {
  __shared__ u32x4 sh[256];
  const int c8 = threadIdx.x & 31, n = a.col0 + blockIdx.x * 256 + 8 * c8;
  const int r0 = (int)((int64_t)blockIdx.y * a.cin / gridDim.y), r1 = (int)((int64_t)(blockIdx.y + 1) * a.cin / gridDim.y);
  u32x4 m = {0u, 0u, 0u, 0u};
  if (n < a.col1)
    for (int r = r0 + (threadIdx.x >> 5); r < r1; r += 8) {
      const u32x4 v = load_row8(a.x + r * a.ldx, n, a.col1);
#pragma unroll
      for (int u = 0; u < 4; ++u) m[u] = fp8_max_finite(m[u], v[u]);
    }
  sh[threadIdx.x] = m;
  __syncthreads();
  if (threadIdx.x < 32 && n < a.col1) {
    for (int k = 1; k < 8; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) m[u] = fp8_max_finite(m[u], sh[32 * k + threadIdx.x][u]);
    *reinterpret_cast<u32x4*>(part + (int64_t)blockIdx.y * a.ld8 + blockIdx.x * 256 + 8 * c8) = m;
  }
}

__global__ __launch_bounds__(256) void fp8_columns_kernel(Fp8Args a, const uint16_t* __restrict__ part, int chunks,
                                                          uint8_t* __restrict__ x8, uint8_t* __restrict__ xs) {
  __shared__ u32x4 sh[256];
  const int c8 = threadIdx.x & 31, k0 = blockIdx.x * 256 + 8 * c8, n = a.col0 + k0;
  const int r0 = (int)((int64_t)blockIdx.y * a.cin / gridDim.y), r1 = (int)((int64_t)(blockIdx.y + 1) * a.cin / gridDim.y);
  u32x4 m = {0u, 0u, 0u, 0u};
  if (n < a.col1)
    for (int k = threadIdx.x >> 5; k < chunks; k += 8) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(part + (int64_t)k * a.ld8 + k0);
#pragma unroll
      for (int u = 0; u < 4; ++u) m[u] = fp8_max_finite(m[u], v[u]);
    }
  sh[threadIdx.x] = m;
  __syncthreads();
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = fp8_max_finite(m[u], sh[32 * k + c8][u]);
  uint32_t e[8];
  float inv[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    e[u] = fp8_scale_of((m[u >> 1] >> (16 * (u & 1))) & 0xffffu);
    inv[u] = fp8_inverse(e[u]);
  }
  if (k0 >= a.ld8) return;
  if (blockIdx.y == 0 && threadIdx.x < 32)
    for (int u = 0; u < 8; ++u) xs[k0 + u] = (uint8_t)e[u];
  for (int r = r0 + (threadIdx.x >> 5); r < r1; r += 8) {
    const u32x4 v = n < a.col1 ? load_row8(a.x + r * a.ldx, n, a.col1) : u32x4{0u, 0u, 0u, 0u};
    fp8_u32x2 c;
    c[0] = fp8_codes<true>(fp8_codes<false>(0u, v[0], inv[0], inv[1]), v[1], inv[2], inv[3]);
    c[1] = fp8_codes<true>(fp8_codes<false>(0u, v[2], inv[4], inv[5]), v[3], inv[6], inv[7]);
    *reinterpret_cast<fp8_u32x2*>(x8 + (int64_t)r * a.ld8 + k0) = c;
  }
}

// Columns [lo, hi) of expert e within the window.
__device__ inline void window_of(const Fp8Args& a, int e, int& lo, int& hi) {
  range_of(a, e, lo, hi);
  lo = max(lo, a.col0);
  hi = max(lo, min(hi, a.col1));
}

// ---------------------------------------------------------------------------
// Simple kernel: 64 rows x 16 tokens of one expert a workgroup, four waves of
// 16 rows; X rows go through LDS element by element.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void fp8_simple_kernel(Fp8Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t xt[64 * 16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, kc = lane >> 4;
  const int nrb = a.rows / 64;
  const int t = blockIdx.x / nrb, rb = blockIdx.x % nrb;
  int first = 0;
  for (int e = 0; e < a.n_experts; ++e) {
    int lo, hi;
    window_of(a, e, lo, hi);
    const int nb = (hi - lo + 15) / 16;
    int tb = (int)((blockIdx.y + gridDim.y - first % gridDim.y) % gridDim.y);
    for (; tb < nb; tb += gridDim.y) {
      const int n0 = lo + tb * 16;
      const float xs = n0 + i16 < hi ? fp8_scale(a.xs[n0 + i16 - a.col0]) : 1.f;
      f32x4 sum = {0.f, 0.f, 0.f, 0.f};
      for (int b = 0; b < a.nkb_d + a.nkb_s; ++b) {
        const bool dense = b < a.nkb_d;
        const int k = dense ? b : b - a.nkb_d;
        const int64_t kb = dense ? (int64_t)t * a.nkb_d + k : (int64_t)t * a.nkb_s + k;
        const int32_t* idx = dense ? a.idx_d + e * a.n_idx_d + kb * 32 : a.idx_s + e * a.n_idx_s + kb * 64;
        // a dense block is multiplied as a 2:4 block whose groups keep positions 0 and 1: column 2 q + u at 4 q + u
        for (int q = threadIdx.x; q < 1024; q += 256) {
          const int p = q / 16, n = q % 16, c = idx[dense ? 2 * (p >> 2) + (p & 1) : p];
          xt[q] = c >= 0 && c < a.cin && n0 + n < hi ? a.x8[(int64_t)c * a.ld8 + n0 + n - a.col0] : (uint8_t)0;
        }
        __syncthreads();
        const int64_t row = kb * a.rows + rb * 64 + wave * 16;
        const uint8_t* val = dense ? a.val_d + e * a.n_val_d : a.val_s + e * a.n_val_s;
        const int64_t group = dense ? (int64_t)t * ((a.nkb_d + 3) / 4) + k / 4 : (int64_t)t * ((a.nkb_s + 3) / 4) + k / 4;
        const uint8_t* sc = (dense ? a.scale_d + e * a.n_scale_d : a.scale_s + e * a.n_scale_s) + group * a.rows + rb * 64 + wave * 16;
        const bf16x8 av = __builtin_bit_cast(bf16x8, fp8_expand(*reinterpret_cast<const fp8_u32x2*>(val + (row + i16) * 32 + 8 * kc), fp8_scale(sc[i16])));
        const int sidx = dense ? 0x4444 : reinterpret_cast<const uint16_t*>(a.meta + e * a.n_meta)[(row + i16) * 4 + kc];
        const uint8_t* bp = xt + (8 * kc + (i16 >> 1)) * 16 + 8 * (i16 & 1);
        const bf16x8 b0 = __builtin_bit_cast(bf16x8, fp8_expand(tr_read8(bp), xs)), b1 = __builtin_bit_cast(bf16x8, fp8_expand(tr_read8(bp + 32 * 16), xs));
        const bf16x16 bv = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
        sum = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av, bv, sum, sidx, 0, 0);
        __syncthreads();
      }
      if (n0 + i16 < hi)
        for (int k = 0; k < 4; ++k)
          a.y[((int64_t)t * a.rows + rb * 64 + wave * 16 + 4 * kc + k) * a.ldy + n0 + i16] = to_bf16(sum[k]);
    }
    first += nb;
  }
}

int check_cols(int64_t n_cols) {
  if (n_cols < 0) return fail(HINM_ESHAPE, "%lld columns", (long long)n_cols);
  if (n_cols > (1 << 24)) return fail(HINM_ESHAPE, "%lld columns exceed 2^24", (long long)n_cols);
  return HINM_OK;
}

int check_args(const hinm_plan_t& p, int32_t n_experts, const void* x, int64_t n_cols, int64_t ldx, const void* y,
               int64_t ldy) {
  if (p.tile_rows % 64 != 0) return fail(HINM_ESHAPE, "tile_rows=%d is not a multiple of 64", p.tile_rows);
  if (n_experts < 1 || n_experts > HINM_MAX_EXPERTS)
    return fail(HINM_ESHAPE, "n_experts=%d; 1 to %d are supported", n_experts, HINM_MAX_EXPERTS);
  const int st = check_cols(n_cols);
  if (st) return st;
  if (ldx < n_cols || ldy < n_cols)
    return fail(HINM_ESHAPE, "ldx=%lld and ldy=%lld must be >= the %lld columns", (long long)ldx, (long long)ldy,
                (long long)n_cols);
  const int64_t lim = (int64_t)1 << 31;
  if (p.bytes_val_dense >= lim || p.bytes_val_24 >= lim || p.bytes_idx_dense >= lim || p.bytes_idx_24 >= lim)
    return fail(HINM_ESHAPE, "each weight's buffers must be below 2^31 bytes");
  if (p.cin > (1 << 22)) return fail(HINM_ESHAPE, "cin=%d exceeds 2^22", p.cin);
  if (n_cols == 0) return HINM_OK;
  if (!x || !y) return fail(HINM_EINVAL, "x and y must be non-NULL");
  if (!hinm::aligned(x, 2) || !hinm::aligned(y, 2)) return fail(HINM_EALIGN, "x and y must be 2-byte aligned");
  return HINM_OK;
}

// Workspace: arrival counters and partial sums, then the rounded activations of
// one window of columns (at most 2^30 bytes, a multiple of 256 columns), their
// scales and the pieces' largest magnitudes.
struct Workspace {
  int64_t window, ld8;               // columns of a window, their pitch
  int64_t x8, xs, part, bytes;       // offsets
  int chunks;
};
Workspace workspace_of(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols) {
  Workspace w{};
  if (n_cols == 0) return w;
  w.window = std::min(n_cols, std::max<int64_t>(256, ((int64_t)1 << 30) / p.cin / 256 * 256));
  w.ld8 = (w.window + 127) / 128 * 128;
  w.chunks = (int)std::min<int64_t>(kChunks, (p.cin + 63) / 64);
  w.x8 = hinm::kWsCounterBytes;
  w.xs = w.x8 + p.cin * w.ld8;
  w.part = w.xs + w.ld8;
  w.bytes = w.part + (int64_t)w.chunks * w.ld8 * 2;
  return w;
}

int launch(const hinm_fp8_t* k, int32_t n_experts, const void* x, int64_t n_cols, int64_t ldx, const int32_t* starts,
           const int32_t* counts, void* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream_) {
  const hinm_plan_t& p = k->plan;
  int st = check_args(p, n_experts, x, n_cols, ldx, y, ldy);
  if (st) return st;
  if (n_cols == 0) return HINM_OK;
  const struct { const void* ptr; int64_t bytes; const char* name; } bufs[7] = {
      {k->val_dense, p.bytes_val_dense, "val_dense"}, {k->scale_dense, p.bytes_val_dense, "scale_dense"},
      {k->idx_dense, p.bytes_idx_dense, "idx_dense"}, {k->val_24, p.bytes_val_24, "val_24"},
      {k->scale_24, p.bytes_val_24, "scale_24"}, {k->meta_24, p.bytes_meta_24, "meta_24"}, {k->idx_24, p.bytes_idx_24, "idx_24"}};
  for (const auto& b : bufs) {
    if (b.bytes > 0 && !b.ptr) return fail(HINM_EINVAL, "%s is NULL but holds %lld bytes", b.name, (long long)b.bytes);
    if (!hinm::aligned(b.ptr, 16)) return fail(HINM_EALIGN, "%s is not 16-byte aligned", b.name);
  }
  const Workspace w = workspace_of(p, n_experts, n_cols);
  if (!workspace || workspace_bytes < (size_t)w.bytes)
    return fail(HINM_EWORKSPACE, "workspace of %zu bytes given, %lld needed", workspace_bytes, (long long)w.bytes);
  if (!hinm::aligned(workspace, 256)) return fail(HINM_EALIGN, "workspace is not 256-byte aligned");
  st = hinm::ensure_device();
  if (st) return st;
  char* const ws = static_cast<char*>(workspace);
  Fp8Args a{};
  a.val_d = k->val_dense;
  a.val_s = k->val_24;
  a.scale_d = k->scale_dense;
  a.scale_s = k->scale_24;
  a.meta = k->meta_24;
  a.idx_d = k->idx_dense;
  a.idx_s = k->idx_24;
  a.nkb_d = p.n_dense_pad / HINM_KB_DENSE;
  a.nkb_s = p.n_24_pad / HINM_KB_24;
  a.n_val_d = p.bytes_val_dense / 2;
  a.n_val_s = p.bytes_val_24 / 2;
  a.n_scale_d = (int64_t)p.cout * ((a.nkb_d + 3) / 4);
  a.n_scale_s = (int64_t)p.cout * ((a.nkb_s + 3) / 4);
  a.n_meta = p.bytes_meta_24 / 8;
  a.n_idx_d = p.bytes_idx_dense / 4;
  a.n_idx_s = p.bytes_idx_24 / 4;
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.x8 = reinterpret_cast<const uint8_t*>(ws + w.x8);
  a.xs = reinterpret_cast<const uint8_t*>(ws + w.xs);
  a.ld8 = (int)w.ld8;
  a.y = static_cast<uint16_t*>(y);
  a.ldy = ldy;
  a.starts = starts;
  a.counts = counts;
  a.n_experts = n_experts;
  a.n_cols = (int)n_cols;
  a.cin = p.cin;
  a.cout = p.cout;
  a.rows = p.tile_rows;
  a.n_tiles = p.n_tiles;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  uint16_t* const part = reinterpret_cast<uint16_t*>(ws + w.part);
  for (int64_t c0 = 0; c0 < n_cols; c0 += w.window) {
    a.col0 = (int)c0;
    a.col1 = (int)std::min(n_cols, c0 + w.window);
    const int cols = a.col1 - a.col0;
    const dim3 grid((unsigned)((cols + 255) / 256), (unsigned)w.chunks);
    hipLaunchKernelGGL(fp8_colmax_kernel, grid, dim3(256), 0, stream, a, part);
    hipLaunchKernelGGL(fp8_columns_kernel, grid, dim3(256), 0, stream, a, part, w.chunks,
                       reinterpret_cast<uint8_t*>(ws + w.x8), reinterpret_cast<uint8_t*>(ws + w.xs));
    const int64_t tbs = cols / 16 + std::min<int64_t>(n_experts, cols) + 1;
    const dim3 g2((unsigned)(p.cout / 64), (unsigned)std::min<int64_t>(tbs, 65535));
    hipLaunchKernelGGL(fp8_simple_kernel, g2, dim3(256), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(HINM_EHIP, "8-bit product launch: %s", hipGetErrorString(e));
  }
  return HINM_OK;
}

}  // namespace

extern "C" int hinm_spmm_experts_fp8_workspace_bytes(const hinm_plan_t* plan, int32_t n_experts, int64_t n_cols,
                                                     size_t* bytes) {
  hinm::clear_error();
  int st = hinm::check_plan(plan);
  if (st) return st;
  st = check_args(*plan, n_experts, nullptr, 0, 0, nullptr, 0);
  if (st) return st;
  if (!bytes) return fail(HINM_EINVAL, "bytes is NULL");
  st = check_cols(n_cols);
  if (st) return st;
  *bytes = (size_t)workspace_of(*plan, n_experts, n_cols).bytes;
  return HINM_OK;
}

extern "C" int hinm_spmm_fp8_workspace_bytes(const hinm_plan_t* plan, int64_t batch, size_t* bytes) {
  return hinm_spmm_experts_fp8_workspace_bytes(plan, 1, batch, bytes);
}

extern "C" int hinm_spmm_experts_fp8(const hinm_fp8_t* stack, int32_t n_experts, const void* x_bf16, int64_t n_cols,
                                     int64_t ldx, const int32_t* starts, const int32_t* counts, void* y_bf16,
                                     int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  hinm::clear_error();
  if (!stack) return fail(HINM_EINVAL, "stack is NULL");
  int st = hinm::check_plan(&stack->plan);
  if (st) return st;
  if (!starts || !counts) return fail(HINM_EINVAL, "starts and counts must be non-NULL");
  if (!hinm::aligned(starts, 4) || !hinm::aligned(counts, 4))
    return fail(HINM_EALIGN, "starts and counts must be 4-byte aligned");
  return launch(stack, n_experts, x_bf16, n_cols, ldx, starts, counts, y_bf16, ldy, workspace, workspace_bytes, stream);
}

extern "C" int hinm_spmm_fp8(const hinm_fp8_t* packed, const void* x_bf16, int64_t batch, int64_t ldx, void* y_bf16,
                             int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  hinm::clear_error();
  if (!packed) return fail(HINM_EINVAL, "packed is NULL");
  int st = hinm::check_plan(&packed->plan);
  if (st) return st;
  return launch(packed, 1, x_bf16, batch, ldx, nullptr, nullptr, y_bf16, ldy, workspace, workspace_bytes, stream);
}
