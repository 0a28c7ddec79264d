// hinm_spmm_experts: one product per expert over its own ragged range of
// columns, Y[:, i] = (W_e (.) M_e) X[:, i], with bf16 or 4-bit microscaled
// packed values; hinm_spmm_mx4 is the same product with one weight and one
// range.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <climits>

#include "hinm_device.h"
#include "hinm_internal.h"
#include "hinm_mx4.h"

using hinm::fail;

namespace {

// The weights of all experts and the activations.  Strides are per expert.
struct ExpArgs {
  const uint8_t *val_d, *val_s;      // bf16 values or codes
  const uint8_t *scale_d, *scale_s;  // 4-bit only
  const uint8_t* meta;               // uint64 a row (bf16) or hinm_mx4_t's order
  const int32_t *idx_d, *idx_s;
  int64_t bytes_val_d, bytes_val_s, bytes_meta, n_idx_d, n_idx_s;   // of one expert
  const uint16_t* x;
  uint16_t* y;
  int64_t ldx, ldy;
  const int32_t *starts, *counts;    // NULL: one range, all columns
  int n_experts, n_cols;
  int cin, cout, rows, n_tiles, nkb_d, nkb_s;
};

// Columns [lo, hi) of expert e, clipped to the buffer.
__device__ inline void range_of(const ExpArgs& a, int e, int& lo, int& hi) {
  if (!a.starts) {
    lo = 0;
    hi = a.n_cols;
    return;
  }
  const int s = a.starts[e], c = a.counts[e];
  lo = min(max(s, 0), a.n_cols);
  hi = s < 0 || c <= 0 ? lo : lo + min(c, a.n_cols - lo);
}

// ---------------------------------------------------------------------------
// General kernel: any alignment, 64-bit addresses.  Workgroup = 64 rows x 16
// tokens of one expert, four waves of 16 rows; X rows go through LDS
// transposed, element by element.
// ---------------------------------------------------------------------------
constexpr int kGenTok = 16;
constexpr int kGenPitch = 72;        // LDS row pitch in bf16 (64 positions + 16 bytes)

template <bool MX4>
__global__ __launch_bounds__(256) void experts_general_kernel(ExpArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t xt[kGenTok * kGenPitch];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i16 = lane & 15, kc = lane >> 4;
  const int nrb = a.rows / 64;
  const int t = blockIdx.x / nrb, rb = blockIdx.x % nrb;
  int first = 0;                     // token blocks of the experts before e
  for (int e = 0; e < a.n_experts; ++e) {
    int lo, hi;
    range_of(a, e, lo, hi);
    const int nb = (hi - lo + kGenTok - 1) / kGenTok;
    // this workgroup's token blocks: those whose number is blockIdx.y mod gridDim.y
    int tb = (int)((blockIdx.y + gridDim.y - first % gridDim.y) % gridDim.y);
    for (; tb < nb; tb += gridDim.y) {
      const int n0 = lo + tb * kGenTok;
      auto gather = [&](const int32_t* idx, int k_n) {
        for (int q = threadIdx.x; q < k_n * kGenTok; q += 256) {
          const int k = q / kGenTok, n = q % kGenTok, c = idx[k];
          xt[n * kGenPitch + k] = c >= 0 && c < a.cin && n0 + n < hi ? a.x[(int64_t)c * a.ldx + n0 + n] : (uint16_t)0;
        }
      };
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      for (int b = 0; b < a.nkb_d + a.nkb_s; ++b) {
        const bool dense = b < a.nkb_d;
        const int64_t kb = dense ? (int64_t)t * a.nkb_d + b : (int64_t)t * a.nkb_s + (b - a.nkb_d);
        if (dense) gather(a.idx_d + e * a.n_idx_d + kb * 32, 32);
        else gather(a.idx_s + e * a.n_idx_s + kb * 64, 64);
        __syncthreads();
        const uint8_t* val = dense ? a.val_d + e * a.bytes_val_d : a.val_s + e * a.bytes_val_s;
        bf16x8 av;
        int sidx = 0;
        if constexpr (MX4) {
          const int64_t u = kb * nrb + rb;
          const int at = i16 * 4 + wave;
          const uint8_t* sc = dense ? a.scale_d + e * (a.bytes_val_d / 16) : a.scale_s + e * (a.bytes_val_s / 16);
          av = mx4_expand(reinterpret_cast<const uint32_t*>(val)[u * 256 + kc * 64 + at], mx4_scale(sc[u * 64 + at]));
          if (!dense) sidx = reinterpret_cast<const uint16_t*>(a.meta + e * a.bytes_meta)[u * 256 + kc * 64 + at];
        } else {
          const int64_t row = kb * a.rows + rb * 64 + wave * 16 + i16;
          av = *reinterpret_cast<const bf16x8*>(val + row * 64 + 16 * kc);
          if (!dense) sidx = reinterpret_cast<const uint16_t*>(a.meta + e * a.bytes_meta)[row * 4 + kc];
        }
        const uint16_t* bp = xt + i16 * kGenPitch + 8 * kc;
        const bf16x8 b0 = *reinterpret_cast<const bf16x8*>(bp);
        if (dense) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, b0, acc, 0, 0, 0);
        } else {
          const bf16x8 b1 = *reinterpret_cast<const bf16x8*>(bp + 32);
          const bf16x16 bv = __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
          acc = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av, bv, acc, sidx, 0, 0);
        }
        __syncthreads();
      }
      if (n0 + i16 < hi)
        for (int k = 0; k < 4; ++k)
          a.y[((int64_t)t * a.rows + rb * 64 + wave * 16 + 4 * kc + k) * a.ldy + n0 + i16] = bf16_rne(acc[k]);
    }
    first += nb;
  }
}

int check_args(const hinm_plan_t& p, int32_t n_experts, const void* x, int64_t n_cols, int64_t ldx, const void* y,
               int64_t ldy) {
  if (p.tile_rows % 64 != 0) return fail(HINM_ESHAPE, "tile_rows=%d is not a multiple of 64", p.tile_rows);
  if (n_experts < 1 || n_experts > HINM_MAX_EXPERTS)
    return fail(HINM_ESHAPE, "n_experts=%d; 1 to %d are supported", n_experts, HINM_MAX_EXPERTS);
  if (n_cols < 0) return fail(HINM_ESHAPE, "%lld columns", (long long)n_cols);
  if (n_cols > (1 << 24)) return fail(HINM_ESHAPE, "%lld columns exceed 2^24", (long long)n_cols);
  if (ldx < n_cols || ldy < n_cols)
    return fail(HINM_ESHAPE, "ldx=%lld and ldy=%lld must be >= the %lld columns", (long long)ldx, (long long)ldy,
                (long long)n_cols);
  const int64_t lim = (int64_t)1 << 31;
  if (p.bytes_val_dense >= lim || p.bytes_val_24 >= lim || p.bytes_idx_dense >= lim || p.bytes_idx_24 >= lim)
    return fail(HINM_ESHAPE, "each weight's buffers must be below 2^31 bytes");
  if (n_cols == 0) return HINM_OK;
  if (!x || !y) return fail(HINM_EINVAL, "x and y must be non-NULL");
  if (!hinm::aligned(x, 2) || !hinm::aligned(y, 2)) return fail(HINM_EALIGN, "x and y must be 2-byte aligned");
  return HINM_OK;
}

struct Buf {
  const void* ptr;
  int64_t bytes;
  const char* name;
};

int check_bufs(const Buf* b, int n) {
  for (int i = 0; i < n; ++i) {
    if (b[i].bytes > 0 && !b[i].ptr)
      return fail(HINM_EINVAL, "%s is NULL but holds %lld bytes", b[i].name, (long long)b[i].bytes);
    if (!hinm::aligned(b[i].ptr, 16)) return fail(HINM_EALIGN, "%s is not 16-byte aligned", b[i].name);
  }
  return HINM_OK;
}

int64_t ws_bytes(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols) {
  (void)p;
  (void)n_experts;
  (void)n_cols;
  return 0;
}

// The product behind every entry point; `a` holds the weights' pointers.
template <bool MX4>
int launch(const hinm_plan_t& p, int32_t n_experts, ExpArgs a, const void* x, int64_t n_cols, int64_t ldx,
           const int32_t* starts, const int32_t* counts, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
           void* stream_) {
  const int64_t need = ws_bytes(p, n_experts, n_cols);
  if (need > 0) {
    if (!workspace || workspace_bytes < (size_t)need)
      return fail(HINM_EWORKSPACE, "workspace of %zu bytes given, %lld needed", workspace_bytes, (long long)need);
    if (!hinm::aligned(workspace, 256)) return fail(HINM_EALIGN, "workspace is not 256-byte aligned");
  }
  const int st = hinm::ensure_device();
  if (st) return st;
  a.x = static_cast<const uint16_t*>(x);
  a.y = static_cast<uint16_t*>(y);
  a.ldx = ldx;
  a.ldy = ldy;
  a.starts = starts;
  a.counts = counts;
  a.n_experts = n_experts;
  a.n_cols = (int)n_cols;
  a.cin = p.cin;
  a.cout = p.cout;
  a.rows = p.tile_rows;
  a.n_tiles = p.n_tiles;
  a.nkb_d = p.n_dense_pad / HINM_KB_DENSE;
  a.nkb_s = p.n_24_pad / HINM_KB_24;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  const int64_t tbs = n_cols / kGenTok + std::min<int64_t>(n_experts, n_cols);
  const dim3 grid((unsigned)(p.cout / 64), (unsigned)std::min<int64_t>(tbs, 65535));
  hipLaunchKernelGGL(experts_general_kernel<MX4>, grid, dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? HINM_OK : fail(HINM_EHIP, "experts launch: %s", hipGetErrorString(e));
}

int check_ranges(const int32_t* starts, const int32_t* counts) {
  if (!starts || !counts) return fail(HINM_EINVAL, "starts and counts must be non-NULL");
  if (!hinm::aligned(starts, 4) || !hinm::aligned(counts, 4))
    return fail(HINM_EALIGN, "starts and counts must be 4-byte aligned");
  return HINM_OK;
}

int run_mx4(const hinm_mx4_t* k, int32_t n_experts, const void* x, int64_t n_cols, int64_t ldx, const int32_t* starts,
            const int32_t* counts, void* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  const hinm_plan_t& p = k->plan;
  int st = check_args(p, n_experts, x, n_cols, ldx, y, ldy);
  if (st) return st;
  const Buf b[7] = {{k->val_dense, p.bytes_val_dense, "val_dense"}, {k->scale_dense, p.bytes_val_dense, "scale_dense"},
                    {k->idx_dense, p.bytes_idx_dense, "idx_dense"}, {k->val_24, p.bytes_val_24, "val_24"},
                    {k->scale_24, p.bytes_val_24, "scale_24"}, {k->meta_24, p.bytes_meta_24, "meta_24"},
                    {k->idx_24, p.bytes_idx_24, "idx_24"}};
  if (n_cols == 0) return HINM_OK;
  st = check_bufs(b, 7);
  if (st) return st;
  ExpArgs a{};
  a.val_d = reinterpret_cast<const uint8_t*>(k->val_dense);
  a.val_s = reinterpret_cast<const uint8_t*>(k->val_24);
  a.scale_d = k->scale_dense;
  a.scale_s = k->scale_24;
  a.meta = reinterpret_cast<const uint8_t*>(k->meta_24);
  a.idx_d = k->idx_dense;
  a.idx_s = k->idx_24;
  a.bytes_val_d = p.bytes_val_dense / 4;
  a.bytes_val_s = p.bytes_val_24 / 4;
  a.bytes_meta = p.bytes_meta_24;
  a.n_idx_d = p.bytes_idx_dense / 4;
  a.n_idx_s = p.bytes_idx_24 / 4;
  return launch<true>(p, n_experts, a, x, n_cols, ldx, starts, counts, y, ldy, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" int hinm_spmm_experts_workspace_bytes(const hinm_plan_t* plan, int32_t n_experts, int64_t n_cols,
                                                 size_t* bytes) {
  hinm::clear_error();
  int st = hinm::check_plan(plan);
  if (st) return st;
  st = check_args(*plan, n_experts, nullptr, 0, 0, nullptr, 0);
  if (st) return st;
  if (!bytes) return fail(HINM_EINVAL, "bytes is NULL");
  if (n_cols < 0) return fail(HINM_ESHAPE, "%lld columns", (long long)n_cols);
  *bytes = (size_t)ws_bytes(*plan, n_experts, n_cols);
  return HINM_OK;
}

extern "C" int hinm_spmm_mx4_workspace_bytes(const hinm_plan_t* plan, int64_t batch, size_t* bytes) {
  return hinm_spmm_experts_workspace_bytes(plan, 1, batch, bytes);
}

extern "C" int hinm_spmm_experts(const hinm_packed_t* stack, int32_t n_experts, const void* x_bf16, int64_t n_cols,
                                 int64_t ldx, const int32_t* starts, const int32_t* counts, void* y_bf16, int64_t ldy,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  hinm::clear_error();
  if (!stack) return fail(HINM_EINVAL, "stack is NULL");
  int st = hinm::check_plan(&stack->plan);
  if (st) return st;
  const hinm_plan_t& p = stack->plan;
  st = check_ranges(starts, counts);
  if (st) return st;
  st = check_args(p, n_experts, x_bf16, n_cols, ldx, y_bf16, ldy);
  if (st) return st;
  const Buf b[5] = {{stack->val_dense, p.bytes_val_dense, "val_dense"}, {stack->idx_dense, p.bytes_idx_dense, "idx_dense"},
                    {stack->val_24, p.bytes_val_24, "val_24"}, {stack->meta_24, p.bytes_meta_24, "meta_24"},
                    {stack->idx_24, p.bytes_idx_24, "idx_24"}};
  if (n_cols == 0) return HINM_OK;
  st = check_bufs(b, 5);
  if (st) return st;
  ExpArgs a{};
  a.val_d = static_cast<const uint8_t*>(stack->val_dense);
  a.val_s = static_cast<const uint8_t*>(stack->val_24);
  a.meta = reinterpret_cast<const uint8_t*>(stack->meta_24);
  a.idx_d = stack->idx_dense;
  a.idx_s = stack->idx_24;
  a.bytes_val_d = p.bytes_val_dense;
  a.bytes_val_s = p.bytes_val_24;
  a.bytes_meta = p.bytes_meta_24;
  a.n_idx_d = p.bytes_idx_dense / 4;
  a.n_idx_s = p.bytes_idx_24 / 4;
  return launch<false>(p, n_experts, a, x_bf16, n_cols, ldx, starts, counts, y_bf16, ldy, workspace, workspace_bytes,
                       stream);
}

extern "C" int hinm_spmm_experts_mx4(const hinm_mx4_t* stack, int32_t n_experts, const void* x_bf16, int64_t n_cols,
                                     int64_t ldx, const int32_t* starts, const int32_t* counts, void* y_bf16,
                                     int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  hinm::clear_error();
  if (!stack) return fail(HINM_EINVAL, "stack is NULL");
  int st = hinm::check_plan(&stack->plan);
  if (st) return st;
  st = check_ranges(starts, counts);
  if (st) return st;
  return run_mx4(stack, n_experts, x_bf16, n_cols, ldx, starts, counts, y_bf16, ldy, workspace, workspace_bytes, stream);
}

extern "C" int hinm_spmm_mx4(const hinm_mx4_t* packed, const void* x_bf16, int64_t batch, int64_t ldx, void* y_bf16,
                             int64_t ldy, void* workspace, size_t workspace_bytes, void* stream) {
  hinm::clear_error();
  if (!packed) return fail(HINM_EINVAL, "packed is NULL");
  int st = hinm::check_plan(&packed->plan);
  if (st) return st;
  return run_mx4(packed, 1, x_bf16, batch, ldx, nullptr, nullptr, y_bf16, ldy, workspace, workspace_bytes, stream);
}
