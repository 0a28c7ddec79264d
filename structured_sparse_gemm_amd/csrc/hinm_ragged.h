// Device helpers of the products over ragged column ranges (not installed).
// `Args` is a kernel's argument struct with the members starts, counts (NULL:
// one range, all columns), n_experts and n_cols.
#ifndef HINM_RAGGED_H_
#define HINM_RAGGED_H_

#include "hinm_device.h"
#include "hinm_internal.h"

namespace {

constexpr int kCus = 256;            // compute units
constexpr int kMaxWgs = 512;         // workgroups of a prefill launch: two a compute unit

// Round to nearest even (the conversion instruction; NaN stays NaN).
__device__ inline uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// 16 bytes at any 2-byte aligned address (one access: the device takes them).
typedef u32x4 any_u32x4 __attribute__((aligned(2)));

// Columns [lo, hi) of expert e, clipped to the buffer.
template <class Args>
__device__ inline void range_of(const Args& a, int e, int& lo, int& hi) {
  if (!a.starts) {
    lo = 0;
    hi = a.n_cols;
    return;
  }
  const int s = a.starts[e], c = a.counts[e];
  lo = min(max(s, 0), a.n_cols);
  hi = s < 0 || c <= 0 ? lo : lo + min(c, a.n_cols - lo);
}

// Blocks of nt columns before every expert, and their number in all; an
// expert's first block starts at its first column rounded down to a multiple
// of `align`.
template <class Args>
__device__ inline int plan_blocks(const Args& a, int nt, int* pre, int align = 1) {
  if (!a.starts) return (a.n_cols + nt - 1) / nt;
  if (threadIdx.x < 64) {
    int carry = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + (int)threadIdx.x;
      int lo = 0, hi = 0;
      if (e < a.n_experts) range_of(a, e, lo, hi);
      const int nb = hi > lo ? (hi - (lo & -align) + nt - 1) / nt : 0;
      int sum = nb;
      for (int d = 1; d < 64; d *= 2) {
        const int v = __shfl_up(sum, d);
        sum += (int)threadIdx.x >= d ? v : 0;
      }
      if (e < a.n_experts) pre[e] = carry + sum - nb;
      carry += __shfl(sum, 63);
    }
    if (threadIdx.x == 0) pre[a.n_experts] = carry;
  }
  __syncthreads();
  return pre[a.n_experts];
}

// The expert that token block q belongs to: the last one with pre[e] <= q
// (an empty expert shares its number with the next).
template <class Args>
__device__ inline int find_expert(const Args& a, const int* pre, int q) {
  if (!a.starts) return 0;
  int n = 0;
  for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
    const int e = e0 + (int)(threadIdx.x & 63);
    const int c = __popcll(__ballot(e < a.n_experts && pre[min(e, a.n_experts)] <= q));
    n += c;
    if (c < 64) break;
  }
  return __builtin_amdgcn_readfirstlane(n - 1);
}

__device__ inline __amdgpu_buffer_rsrc_t buffer(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)(uint32_t)bytes, kBufferWord3);
}

// Partial sums of a split item: agent-scope stores and loads, as arrive()
// explains; part[(item * splits + split)][n], added in split order by the last
// workgroup to arrive.
template <int N>
__device__ inline bool join_splits(float (&v)[N], float* part, unsigned* counters, int item, int split, int splits,
                                   int* s_last) {
  float* my = part + (int64_t)(item * splits + split) * N * 256 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < N; ++k) __hip_atomic_store(my + k * 256, v[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) *s_last = arrive(counters + item, splits);
  __syncthreads();
  if (!*s_last) return false;
  const float* p0 = part + (int64_t)item * splits * N * 256 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  constexpr int U = N <= 8 ? 4 : 1;                // splits whose loads are in flight at once (one by one: +0.5 us)
  for (int s = 0; s < splits; s += U) {
    float t[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k)
        t[u][k] = __hip_atomic_load(p0 + (int64_t)min(s + u, splits - 1) * N * 256 + k * 256, __ATOMIC_RELAXED,
                                    __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] += s + u < splits ? t[u][k] : 0.f;
  }
  return true;
}

}  // namespace

#endif  // HINM_RAGGED_H_
