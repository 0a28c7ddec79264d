// hinm_spmm_experts: one product per expert over its own ragged range of
// columns, Y[:, i] = (W_e (.) M_e) X[:, i], with bf16 or 4-bit microscaled
// packed values; hinm_spmm_mx4 is the same product with one weight and one
// range.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "hinm_device.h"
#include "hinm_internal.h"
#include "hinm_mx4.h"

using hinm::fail;

namespace {

// Round to nearest even (the conversion instruction; NaN stays NaN).
__device__ inline uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }

// 16 bytes at any 2-byte aligned address (one access: the device takes them).
typedef u32x4 any_u32x4 __attribute__((aligned(2)));

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
  int x_end;                         // 1: the buffer of X ends with row cin - 1's last column (0: its rows are padded)
  int may_split;                     // the workspace has room for arrival counters and partial sums
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
          a.y[((int64_t)t * a.rows + rb * 64 + wave * 16 + 4 * kc + k) * a.ldy + n0 + i16] = to_bf16(acc[k]);
    }
    first += nb;
  }
}

// ---------------------------------------------------------------------------
// Schedule shared by the fast kernels.  The ranges are known on the device
// only, so every workgroup works out the same schedule from them: range e is
// cut into ceil(n_e / NT) token blocks, numbered through all experts
// (pre[e] = blocks before expert e), and an item is one token block times one
// 64-row block.  When the items leave workgroups idle, each item's K-blocks
// are dealt to `splits` workgroups and the partial sums meet in the workspace;
// never where the host, which does not know the ranges, gave it no room for
// them (may_split).
// ---------------------------------------------------------------------------
constexpr int kCus = 256;            // compute units
constexpr int kMaxWgs = 512;         // workgroups of a prefill launch: two a compute unit

__device__ inline int plan_blocks(const ExpArgs& a, int nt, int* pre) {
  if (!a.starts) return (a.n_cols + nt - 1) / nt;
  if (threadIdx.x < 64) {
    int carry = 0;
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + (int)threadIdx.x;
      int lo = 0, hi = 0;
      if (e < a.n_experts) range_of(a, e, lo, hi);
      const int nb = (hi - lo + nt - 1) / nt;
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
__device__ inline int find_expert(const ExpArgs& a, const int* pre, int q) {
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

__device__ inline void x_buffer(const ExpArgs& a, __amdgpu_buffer_rsrc_t& x) {
  x = buffer(a.x, ((int64_t)(a.cin - 1) * a.ldx + (a.x_end ? a.n_cols : a.ldx)) * 2);
}

// The buffer of X ends with its last row's last column, and the range check
// of a buffer load zeroes a dword that crosses the end: with an odd number of
// elements from a chunk's start to that end, the very last element would read
// as zero.  Whoever stages that element (row cin - 1, column n_cols - 1)
// writes its value, read alone, over it.
__device__ inline uint16_t last_element(const ExpArgs& a) { return a.x[(int64_t)(a.cin - 1) * a.ldx + a.n_cols - 1]; }

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

// ---------------------------------------------------------------------------
// Few tokens an expert.  Workgroup = 64 rows x NT tokens; its four waves deal
// the K-blocks among themselves and each works alone - 64 rows x NT tokens of
// its blocks - so the main loop has no barrier: index words are loaded two
// blocks ahead, X rows, values and metadata one block ahead, and X rows pass
// through the wave's own LDS slot for the transposed reads.  At the end the
// waves' sums meet in LDS, in wave order.
//
// What hides the latency of the index -> X row chain is other waves: five
// workgroups a compute unit at 16 tokens (88 VGPRs), four at 32.  With two and
// four blocks in flight and fewer workgroups the same loop was slower (8
// experts of 11008x4096, 4-bit: 34 and 39 us against 32).  At 16 tokens a
// gathered X row is 32 bytes that take a 128-byte line of the load path, 64 of
// the 80 lines of a 4-bit 2:4 block: that path, not memory, bounds the 4-bit
// product (29 us); with bf16 values it is the packed bytes (209 MB in 52 us, 4.0
// TB/s from memory, in 40 partly from the last-level cache).  X held whole in
// LDS removes those lines but leaves one workgroup a unit: 41 us.
// ---------------------------------------------------------------------------
constexpr int decode_wgs(int nt) { return nt == 16 ? 5 : 4; }   // workgroups a compute unit

template <int NT>
__device__ inline int x_granule(int p, int g) {     // 32-byte granule of position p, 16 tokens g; conflict-free
  if constexpr (NT == 16) return p ^ (((p >> 3) & 1) << 2);
  else return 2 * p + (g ^ ((p >> 3) & 1));
}

// One block's values and metadata of one lane: 64 rows' fragments f = 0..3.
template <bool MX4>
struct DecA {
  u32x4 v[4];
  uint32_t m[4];
};
template <>
struct DecA<true> {
  u32x4 v;                 // the codes of the four fragments
  uint32_t scale;
  uint32_t m[2];
};
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool MX4, int NT>
__global__ __launch_bounds__(256, decode_wgs(NT)) void experts_decode_kernel(ExpArgs a,
                                                                                   float* __restrict__ part,
                                                                                   unsigned* __restrict__ counters) {
  constexpr int NB = NT / 16;
  constexpr int XL = NT / 8;                       // X loads a lane for 64 positions
  constexpr int kRed = NT == 16 ? 20 : 34;         // row pitch of the waves' sums (floats); 34: 40 KB of LDS in all
  __shared__ __attribute__((aligned(16))) union {
    uint16_t xs[4][64 * NT];
    float red[4][64 * kRed];
  } sh;
  __shared__ int pre[HINM_MAX_EXPERTS + 1];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i16 = lane & 15, kc = lane >> 4;
  const int nrb = a.rows / 64, n_rb = a.n_tiles * nrb, nblk = a.nkb_d + a.nkb_s;
  uint16_t* const xs = sh.xs[wave];

  const int items = plan_blocks(a, NT, pre) * n_rb;
  // A split costs its row blocks a round trip through the workspace (about 2.5
  // us), so one is made only where compute units would have no item, and for
  // at least four K-blocks a wave (4-bit, 1 token: 4096x11008 9.5 us with
  // four splits of its 64 row blocks and slower with eight, 11.2 against 10.4
  // before the join had several shares in flight; 11008x4096's 172 row blocks
  // 8.3 us whole, 10.6 in two).
  int splits = 1;
  while (a.may_split && items * splits * 2 <= kCus && nblk >= 32 * splits) splits *= 2;

  // A dense block is multiplied as a 2:4 block whose groups keep positions 0
  // and 1: its column 2 q + u sits at position 4 q + u, and positions 4 q + 2
  // and 4 q + 3 hold zeros.  Byte offset in its index list by position, and a
  // mask that makes the index of a position without a column -1:
  const uint32_t l_dense = (lane & 2) ? 0u : 4u * (2 * (lane >> 2) + (lane & 1));
  const int no_index = (lane & 2) ? -1 : 0;
  // this lane's share of a block's X rows: position and first token of load j
  int xpos[XL], xtok[XL];
#pragma unroll
  for (int j = 0; j < XL; ++j) {
    const int chunk = 64 * j + lane, s = chunk >> 1;
    int p, g;
    if constexpr (NT == 16) p = s ^ (((s >> 3) & 1) << 2), g = 0;
    else p = s >> 1, g = (s & 1) ^ ((p >> 3) & 1);
    xpos[j] = p;
    xtok[j] = 16 * g + 8 * (chunk & 1);
  }
  int ro[4][NB];                                   // transposed reads: positions 8 kc + i16 / 4 + {0, 4, 32, 36}
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
      ro[k][nb] = x_granule<NT>(8 * kc + (i16 >> 2) + 4 * (k & 1) + 32 * (k >> 1), nb) * 16 + 4 * (i16 & 3);

  __amdgpu_buffer_rsrc_t rx;
  x_buffer(a, rx);
  const uint32_t ldx_bytes = (uint32_t)a.ldx * 2u;

  for (int work = blockIdx.x; work < items * splits; work += gridDim.x) {
    const int item = work / splits, split = work % splits;
    const int tb = item / n_rb, trb = item % n_rb, t = trb / nrb, rb = trb % nrb;
    const int e = find_expert(a, pre, tb);
    int lo, hi;
    range_of(a, e, lo, hi);
    const int n0 = lo + (tb - (a.starts ? pre[e] : 0)) * NT;
    const __amdgpu_buffer_rsrc_t rvd = buffer(a.val_d + e * a.bytes_val_d, a.bytes_val_d);
    const __amdgpu_buffer_rsrc_t rvs = buffer(a.val_s + e * a.bytes_val_s, a.bytes_val_s);
    const __amdgpu_buffer_rsrc_t rm = buffer(a.meta + e * a.bytes_meta, a.bytes_meta);
    const __amdgpu_buffer_rsrc_t rid = buffer(a.idx_d + e * a.n_idx_d, a.n_idx_d * 4);
    const __amdgpu_buffer_rsrc_t ris = buffer(a.idx_s + e * a.n_idx_s, a.n_idx_s * 4);
    __amdgpu_buffer_rsrc_t rsd, rss;
    if constexpr (MX4) {
      rsd = buffer(a.scale_d + e * (a.bytes_val_d / 16), a.bytes_val_d / 16);
      rss = buffer(a.scale_s + e * (a.bytes_val_s / 16), a.bytes_val_s / 16);
    }
    uint32_t xcol[XL];                             // byte offset in a row, past the buffer for tokens past the range
    // the loads that hold column n_cols - 1 (a lane's loads may be of several positions), as bits, and that
    // column's place in such a load
    uint32_t lastj = 0;
    const int last_at = (a.n_cols - 1 - n0) & 7;
#pragma unroll
    for (int j = 0; j < XL; ++j) {
      const int n = n0 + xtok[j];
      xcol[j] = n < hi ? (uint32_t)n * 2u : 0x80000000u;
      if (n <= a.n_cols - 1 && n + 8 > a.n_cols - 1) lastj |= 1u << j;
    }
    const bool touch = n0 + NT >= a.n_cols;
    const uint16_t xlast = touch ? last_element(a) : (uint16_t)0;

    // worker v of nw takes blocks v, v + nw, ...
    const int v = split * 4 + wave, nw = splits * 4;
    const int cnt = v < nblk ? (nblk - v + nw - 1) / nw : 0;

    f32x4 acc[4][NB];
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) acc[f][nb] = f32x4{0.f, 0.f, 0.f, 0.f};
    // D blocks are in flight; the loops over them stay loops until late in the compiler, which otherwise peels the
    // first block's work into a copy of its own (0.7 us an item)
    constexpr int D = 1;
    DecA<MX4> A[D];
    u32x4 X[D][XL];
    int I[D];
    uint32_t P[D];                                    // loads that hold the buffer's last element

    // Block i of this worker.  A block's place in the packed bytes is a scalar
    // offset and the lane's share a constant.  Past the end the last block is
    // read again (it is in the caches) and its X rows are zeros, so that the
    // loop below has no conditions: every wait is for a known number of
    // younger loads, and a remainder needs no second copy of the code.
    auto block = [&](int i) { return v < nblk ? v + nw * min(i, cnt - 1) : 0; };
    auto load_idx = [&](int i) -> int {
      const int b = block(i);
      const bool dense = b < a.nkb_d;
      const uint32_t kb = dense ? (uint32_t)(t * a.nkb_d + b) : (uint32_t)(t * a.nkb_s + b - a.nkb_d);
      return (int)__builtin_amdgcn_raw_buffer_load_b32(dense ? rid : ris, dense ? l_dense : 4u * lane,
                                                       kb * (dense ? 128u : 256u), 0);
    };
    auto load_a = [&](int i, DecA<MX4>& A) {
      const int b = block(i);
      const bool dense = b < a.nkb_d;
      const uint32_t kb = dense ? (uint32_t)(t * a.nkb_d + b) : (uint32_t)(t * a.nkb_s + b - a.nkb_d);
      const __amdgpu_buffer_rsrc_t rv = dense ? rvd : rvs;
      const uint32_t u = kb * (uint32_t)nrb + rb, um = dense ? 0u : u * 512u;   // a dense block's metadata is not used
      if constexpr (MX4) {
        A.v = __builtin_amdgcn_raw_buffer_load_b128(rv, 256u * kc + 16u * i16, u * 1024u, 0);
        A.scale = __builtin_amdgcn_raw_buffer_load_b32(dense ? rsd : rss, 4u * i16, u * 64u, 0);
        const u32x2 m = __builtin_amdgcn_raw_buffer_load_b64(rm, 128u * kc + 8u * i16, um, 0);
        A.m[0] = m[0];
        A.m[1] = m[1];
      } else {
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          A.v[f] = __builtin_amdgcn_raw_buffer_load_b128(rv, 64u * i16 + 16u * kc + 1024u * f, u * 4096u, 0);
          A.m[f] = __builtin_amdgcn_raw_buffer_load_b16(rm, 8u * i16 + 2u * kc + 128u * f, um, 0);
        }
      }
    };
    // X rows of block i from its index word
    auto load_x = [&](int i, int iw, u32x4 (&x)[XL], uint32_t& p) {
      iw = i < cnt ? iw | (block(i) < a.nkb_d ? no_index : 0) : -1;
      p = 0;
#pragma unroll
      for (int j = 0; j < XL; ++j) {
        const int c = __shfl(iw, xpos[j]);
        x[j] = __builtin_amdgcn_raw_buffer_load_b128(rx, c >= 0 ? __umul24((uint32_t)c, ldx_bytes) + xcol[j] : kOob, 0, 0);
        if (touch) p |= c == a.cin - 1 ? lastj & (1u << j) : 0u;
      }
    };
    auto compute = [&](int i, const DecA<MX4>& A, const u32x4 (&x)[XL], uint32_t p) {
      const bool dense = block(i) < a.nkb_d;
#pragma unroll
      for (int j = 0; j < XL; ++j) *reinterpret_cast<u32x4*>(xs + 8 * (64 * j + lane)) = x[j];
      if (touch) {
#pragma unroll
        for (int j = 0; j < XL; ++j)
          if (p & (1u << j)) xs[8 * (64 * j + lane) + last_at] = xlast;
      }
      __builtin_amdgcn_wave_barrier();
      bf16x8 av[4];
      int sidx[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if constexpr (MX4) {
          av[f] = mx4_expand(A.v[f], mx4_scale((A.scale >> (8 * f)) & 255u));
          sidx[f] = (int)((A.m[f >> 1] >> (16 * (f & 1))) & 0xffffu);
        } else {
          av[f] = __builtin_bit_cast(bf16x8, A.v[f]);
          sidx[f] = (int)A.m[f];
        }
        sidx[f] = dense ? 0x4444 : sidx[f];
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const v4i16 b0 = tr_read(xs + ro[0][nb]), b1 = tr_read(xs + ro[1][nb]);
        const v4i16 b2 = tr_read(xs + ro[2][nb]), b3 = tr_read(xs + ro[3][nb]);
        const bf16x8 lo8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
        const bf16x8 hi8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(b2, b3, 0, 1, 2, 3, 4, 5, 6, 7));
        const bf16x16 bv = __builtin_shufflevector(lo8, hi8, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f][nb] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av[f], bv, acc[f][nb], sidx[f], 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
    };

#pragma unroll
    for (int k = 0; k < D; ++k) I[k] = load_idx(k);
#pragma unroll
    for (int k = 0; k < D; ++k) load_a(k, A[k]);
#pragma unroll
    for (int k = 0; k < D; ++k) {
      load_x(k, I[k], X[k], P[k]);
      I[k] = load_idx(k + D);
    }
    for (int i = 0; i < cnt; i += D) {
#pragma unroll
      for (int k = 0; k < D; ++k) {
        compute(i + k, A[k], X[k], P[k]);
        load_a(i + k + D, A[k]);
        load_x(i + k + D, I[k], X[k], P[k]);
        I[k] = load_idx(i + k + 2 * D);
      }
    }

    // the waves' sums, added in wave order; acc[f][nb][q] is row 16 f + 4 kc + q, token 16 nb + i16
    __syncthreads();
#pragma unroll
    for (int f = 0; f < 4; ++f)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int q = 0; q < 4; ++q) sh.red[wave][(16 * f + 4 * kc + q) * kRed + 16 * nb + i16] = acc[f][nb][q];
    __syncthreads();
    constexpr int OUT = NT / 4;                    // outputs a thread: row threadIdx.x / 4, OUT adjacent tokens
    const int row = threadIdx.x >> 2, col = (threadIdx.x & 3) * OUT;
    float sum[OUT];
#pragma unroll
    for (int q = 0; q < OUT; ++q) {
      const int at = row * kRed + col + q;
      sum[q] = sh.red[0][at] + sh.red[1][at] + sh.red[2][at] + sh.red[3][at];
    }
    if (splits == 1 || join_splits(sum, part, counters, item, split, splits, &s_last)) {
      uint16_t* dst = a.y + ((int64_t)t * a.rows + rb * 64 + row) * a.ldy + n0 + col;
#pragma unroll
      for (int q = 0; q < OUT; ++q)
        if (n0 + col + q < hi) dst[q] = to_bf16(sum[q]);
    }
    __syncthreads();                               // the sums share LDS with the next item's X rows
  }
}

// ---------------------------------------------------------------------------
// Many tokens an expert: bound by the gathered X rows on their way through
// the L2 caches.  Workgroup = 64 rows x NT tokens, four waves of 64 rows x
// NT / 4 tokens.  X rows go straight from memory into a double-buffered LDS
// tile (one block ahead); values follow through registers and LDS (four
// blocks ahead), 4-bit ones becoming bf16 on the way, once a workgroup.  The
// regions' loops are separate, dense on 32x32x16 MFMA, 2:4 on 32x32x32 SMFMAC.
//
// 8 experts of 4096x11008, 4094 columns, bf16: 258-279 us, 3.9 GB of lines from L2
// with 64 of them in flight a compute unit at a mean 330 cycles, which is all
// a unit holds.  One 4-bit weight of 11008x4096, 2047 tokens: 123 us with the
// copy of X (10); 17 lines in flight, the step's barrier and the expansion
// bound it, and 1376 items on 512 workgroups leave a tenth idle at the end.
//
// An XCD takes a contiguous range of the items, row blocks fastest, so its
// workgroups share one token block's X rows in its L2.
//
// Tile layout: position p's row of 2 NT bytes, its 16-byte chunk c at chunk
// c ^ 4 (p % 4), so that a 32-lane half of a transposed read covers every bank
// once.
// ---------------------------------------------------------------------------
// Vector-memory instructions do not move across; everything else may.
__device__ inline void vmem_fence() { __builtin_amdgcn_sched_barrier(0x78f); }

template <bool MX4>
struct PreA {
  typename std::conditional<MX4, uint32_t, u32x4>::type v;   // 8 values of a row
  uint32_t scale;                                            // 4-bit: the row's scale byte
  uint32_t m;                                                // threads 0..127: a dword of the block's metadata
};

template <int NT>
struct Pre {
  static constexpr int TW = NT / 4;            // tokens of a wave
  static constexpr int NTB = TW / 32;          // 32-token tiles of a wave
  static constexpr int CPR = NT / 8;           // 16-byte chunks of a row
  static constexpr int TILE = 64 * NT * 2;     // bytes of an X tile
};

template <bool MX4, int NT, bool DENSE, bool LAST>
__device__ inline void prefill_region(const ExpArgs& a, uint8_t* x0, uint8_t* x1, uint8_t* a0, uint8_t* a1,
                                      uint32_t* m0, uint32_t* m1, __amdgpu_buffer_rsrc_t rx, __amdgpu_buffer_rsrc_t rv,
                                      __amdgpu_buffer_rsrc_t rs, __amdgpu_buffer_rsrc_t rm, __amdgpu_buffer_rsrc_t ri,
                                      int kbase, int nb, int rot, int rb, int n0, int hi, uint16_t xlast,
                                      f32x16 (&acc)[2][Pre<NT>::NTB]) {
  using C = Pre<NT>;
  constexpr int KPOS = DENSE ? 32 : 64;        // positions of a block
  constexpr int RPW = KPOS / 4;                // positions a wave stages
  constexpr int RPL = 64 / C::CPR;             // positions of one load
  constexpr int NJ = RPW / RPL;                // X loads of a wave
  constexpr int XROW = 2 * NT;
  if (nb == 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tok_w = wave * C::TW;
  const int g = lane >> 4, i = lane & 15, kcb = g >> 1, kca = lane >> 5, m32 = lane & 31;
  const int q = lane / C::CPR, sl = lane % C::CPR;
  const int nrb = a.rows / 64;
  const uint32_t ldx_bytes = (uint32_t)a.ldx * 2u;
  uint32_t xoff[NJ];                           // source bytes in a row; past the buffer for tokens past the range
  int xn[NJ];                                  // first token of the chunk
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    xn[j] = n0 + 8 * (sl ^ (4 * ((j * RPL + q) & 3)));
    xoff[j] = xn[j] < hi ? (uint32_t)xn[j] * 2u : 0x80000000u;
  }
  const uint32_t ipos = (uint32_t)(wave * RPW + (lane % RPW));
  auto block = [&](int b) -> uint32_t {        // the order starts at block rot and wraps around
    b = min(b, nb - 1) + rot;
    return (uint32_t)(kbase + (b < nb ? b : b - nb));
  };
  auto load_idx = [&](int b) -> int {
    return (int)__builtin_amdgcn_raw_buffer_load_b32(ri, (block(b) * KPOS + ipos) * 4u, 0, 0);
  };
  auto spread_idx = [&](int iw, int (&ci)[NJ]) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      int c = __builtin_amdgcn_readlane(iw, j * RPL);
#pragma unroll
      for (int u = 1; u < RPL; ++u) {
        const int m = -(int)(q == u);            // a mask: a select would become a branch around the readlane
        c = (c & ~m) | (__builtin_amdgcn_readlane(iw, j * RPL + u) & m);
      }
      ci[j] = c;
    }
  };
  auto load_x = [&](const int (&ci)[NJ], uint8_t* xs) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      load_lds16(rx, xs + (wave * RPW + j * RPL) * XROW, ci[j] < 0 ? kOob : __umul24((uint32_t)ci[j], ldx_bytes) + xoff[j]);
  };
  auto patch_x = [&](const int (&ci)[NJ], uint8_t* xs) {   // the buffer's last element, see last_element()
    if constexpr (LAST) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (ci[j] == a.cin - 1 && xn[j] <= a.n_cols - 1 && xn[j] + 8 > a.n_cols - 1)
          reinterpret_cast<uint16_t*>(xs + (wave * RPW + j * RPL) * XROW)[8 * lane + a.n_cols - 1 - xn[j]] = xlast;
    }
  };
  // the row and chunk of 8 values that this thread brings: in the order of the packed bytes
  const int arow = MX4 ? 16 * (threadIdx.x & 3) + ((threadIdx.x >> 2) & 15) : threadIdx.x >> 2;
  const int achk = MX4 ? wave : threadIdx.x & 3;
  const int aofs = arow * 64 + 16 * (achk ^ ((arow >> 2) & 3));
  constexpr int PA = (MX4 ? 3 : 2) + (DENSE ? 0 : 1);       // loads a step issues after its X rows
  auto load_a = [&](int b, PreA<MX4>& A) {
    const uint32_t kb = block(b);
    if constexpr (MX4) {
      const uint32_t u = kb * (uint32_t)nrb + rb;
      A.v = __builtin_amdgcn_raw_buffer_load_b32(rv, u * 1024u + 4u * threadIdx.x, 0, 0);
      A.scale = __builtin_amdgcn_raw_buffer_load_b8(rs, u * 64u + lane, 0, 0);
      if constexpr (!DENSE)
        A.m = __builtin_amdgcn_raw_buffer_load_b32(rm, threadIdx.x < 128 ? u * 512u + 4u * threadIdx.x : kOob, 0, 0);
    } else {
      const uint32_t row = kb * (uint32_t)a.rows + rb * 64u;
      A.v = __builtin_amdgcn_raw_buffer_load_b128(rv, row * 64u + 16u * threadIdx.x, 0, 0);
      if constexpr (!DENSE)
        A.m = __builtin_amdgcn_raw_buffer_load_b32(rm, threadIdx.x < 128 ? row * 8u + 4u * threadIdx.x : kOob, 0, 0);
    }
  };
  auto store_a = [&](uint8_t* as, uint32_t* ms, const PreA<MX4>& A) {
    if constexpr (MX4) *reinterpret_cast<bf16x8*>(as + aofs) = mx4_expand(A.v, mx4_scale(A.scale));
    else *reinterpret_cast<u32x4*>(as + aofs) = A.v;
    if constexpr (!DENSE)
      if (threadIdx.x < 128) ms[threadIdx.x] = A.m;
  };
  const uint32_t cb0 = (uint32_t)(tok_w / 8 + 2 * (g & 1) + ((i >> 1) & 1));
  const uint32_t bsw = (uint32_t)(4 * ((i >> 2) & 3));
  auto compute = [&](const uint8_t* xb, const uint8_t* as, const uint32_t* ms) {
    bf16x8 av[2][2];
    int sidx[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 32 * r + m32;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int q = 2 * s + kca;             // values and metadata 8q.. of the row
        av[r][s] = *reinterpret_cast<const bf16x8*>(as + row * 64 + 16 * (q ^ ((row >> 2) & 3)));
        if constexpr (!DENSE)
          sidx[r][s] = (int)reinterpret_cast<const uint16_t*>(ms)[MX4 ? q * 64 + (row & 15) * 4 + (row >> 4) : row * 4 + q];
      }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < C::NTB; ++j) {
        const uint8_t* base = xb + 16u * ((cb0 + 4u * j) ^ bsw) + 8u * (i & 1) +
                              ((DENSE ? 16 : 32) * s + 8 * kcb + (i >> 2)) * XROW;
        const v4i16 b0 = tr_read_b(base), b1 = tr_read_b(base + 4 * XROW);
        const bf16x8 lo8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7));
        if constexpr (DENSE) {
#pragma unroll
          for (int r = 0; r < 2; ++r)
            acc[r][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(av[r][s], lo8, acc[r][j], 0, 0, 0);
        } else {
          const v4i16 b2 = tr_read_b(base + 16 * XROW), b3 = tr_read_b(base + 20 * XROW);
          const bf16x8 hi8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(b2, b3, 0, 1, 2, 3, 4, 5, 6, 7));
          const bf16x16 bv = __builtin_shufflevector(lo8, hi8, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
          for (int r = 0; r < 2; ++r)
            acc[r][j] = __builtin_amdgcn_smfmac_f32_32x32x32_bf16(av[r][s], bv, acc[r][j], sidx[r][s], 0, 0);
        }
      }
  };

  uint8_t* const xt[2] = {x0, x1};
  uint8_t* const at[2] = {a0, a1};
  uint32_t* const mt[2] = {m0, m1};
  // Register sets by block number: values of four blocks (block b's are free
  // once they are in LDS, at step b - 1), index words and spread indices of two.
  constexpr int AHEAD = 4;
  PreA<MX4> A[AHEAD];
  int Iw[2], CI[2][NJ];
  __syncthreads();                             // the tiles may still be read by the previous region
  Iw[0] = load_idx(0);
  Iw[1] = load_idx(1);
#pragma unroll
  for (int d = 0; d < AHEAD; ++d) load_a(d, A[d]);
  spread_idx(Iw[0], CI[0]);
  spread_idx(Iw[1], CI[1]);
  load_x(CI[0], xt[0]);
  vmem_fence();                                // wait_vm counts the loads behind the X rows
  Iw[0] = load_idx(2);
  store_a(at[0], mt[0], A[0]);
  vmem_fence();
  wait_vm<1>();                                // block 0's X rows
  patch_x(CI[0], xt[0]);
  __syncthreads();
  // Step b: X rows of b + 1 into the other tile, index word of b + 3, values
  // of b + AHEAD; multiply b; the values of b + 1 into LDS; wait for the X rows.
  auto step = [&](auto kk, int b) {
    constexpr int k = decltype(kk)::value, k2 = k % 2;
    __builtin_amdgcn_s_setprio(2);             // the loads go out ahead of the other workgroup's arithmetic
    if (b + 1 < nb) load_x(CI[1 - k2], xt[1 - k2]);
    vmem_fence();
    Iw[1 - k2] = load_idx(b + 3);
    load_a(b + AHEAD, A[k]);
    vmem_fence();
    __builtin_amdgcn_s_setprio(0);
    compute(xt[k2], at[k2], mt[k2]);
    store_a(at[1 - k2], mt[1 - k2], A[(k + 1) % 4]);
    spread_idx(Iw[k2], CI[k2]);                // indices of b + 2
    vmem_fence();
    wait_vm<PA>();
    if (b + 1 < nb) patch_x(CI[1 - k2], xt[1 - k2]);
    __syncthreads();
  };
  int b = 0;
  for (; b + 4 <= nb; b += 4) {
    step(std::integral_constant<int, 0>{}, b);
    step(std::integral_constant<int, 1>{}, b + 1);
    step(std::integral_constant<int, 2>{}, b + 2);
    step(std::integral_constant<int, 3>{}, b + 3);
  }
  if (b < nb) step(std::integral_constant<int, 0>{}, b);
  if (b + 1 < nb) step(std::integral_constant<int, 1>{}, b + 1);
  if (b + 2 < nb) step(std::integral_constant<int, 2>{}, b + 2);
}

template <bool MX4, int NT>
__global__ __launch_bounds__(256, 2) void experts_prefill_kernel(ExpArgs a, float* __restrict__ part,
                                                                 unsigned* __restrict__ counters) {
  using C = Pre<NT>;
  // separate LDS objects: loads into one tile never hold up reads of the other
  __shared__ __attribute__((aligned(16))) uint8_t xs_a[C::TILE];
  __shared__ __attribute__((aligned(16))) uint8_t xs_b[C::TILE];
  __shared__ __attribute__((aligned(16))) uint8_t as_a[64 * 64];
  __shared__ __attribute__((aligned(16))) uint8_t as_b[64 * 64];
  __shared__ __attribute__((aligned(16))) uint32_t ms_a[128];
  __shared__ __attribute__((aligned(16))) uint32_t ms_b[128];
  __shared__ int pre[HINM_MAX_EXPERTS + 1];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nrb = a.rows / 64, n_rb = a.n_tiles * nrb;
  const int tok_w = wave * C::TW;

  const int items = plan_blocks(a, NT, pre) * n_rb;
  int splits = 1;
  while (a.may_split && splits < 4 && items * splits * 2 <= (int)gridDim.x && a.nkb_d + 2 * a.nkb_s >= 16 * splits)
    splits *= 2;
  const int xcd = blockIdx.x % 8, slot = blockIdx.x / 8, per_xcd = gridDim.x / 8;
  const int w_lo = (int)((int64_t)xcd * items * splits / 8), w_hi = (int)((int64_t)(xcd + 1) * items * splits / 8);
  __amdgpu_buffer_rsrc_t rx;
  x_buffer(a, rx);

  for (int work = w_lo + slot; work < w_hi; work += per_xcd) {
    const int item = work / splits, split = work % splits;
    const int tb = item / n_rb, trb = item % n_rb, t = trb / nrb, rb = trb % nrb;
    const int e = find_expert(a, pre, tb);
    int lo, hi;
    range_of(a, e, lo, hi);
    const int n0 = lo + (tb - (a.starts ? pre[e] : 0)) * NT;
    const __amdgpu_buffer_rsrc_t rvd = buffer(a.val_d + e * a.bytes_val_d, a.bytes_val_d);
    const __amdgpu_buffer_rsrc_t rvs = buffer(a.val_s + e * a.bytes_val_s, a.bytes_val_s);
    const __amdgpu_buffer_rsrc_t rm = buffer(a.meta + e * a.bytes_meta, a.bytes_meta);
    const __amdgpu_buffer_rsrc_t rid = buffer(a.idx_d + e * a.n_idx_d, a.n_idx_d * 4);
    const __amdgpu_buffer_rsrc_t ris = buffer(a.idx_s + e * a.n_idx_s, a.n_idx_s * 4);
    const __amdgpu_buffer_rsrc_t rsd = buffer(a.scale_d + e * (a.bytes_val_d / 16), MX4 ? a.bytes_val_d / 16 : 0);
    const __amdgpu_buffer_rsrc_t rss = buffer(a.scale_s + e * (a.bytes_val_s / 16), MX4 ? a.bytes_val_s / 16 : 0);
    // the token block that holds the buffer's last element, where a 4-byte load of a chunk may cross the end; its
    // own instantiation: the check costs 11% (11008x4096, 2048 tokens: 104 -> 117 us with it in every block)
    const bool touch = n0 + NT >= a.n_cols && ((a.n_cols - n0) & 1) && a.x_end;
    const uint16_t xlast = touch ? last_element(a) : (uint16_t)0;

    f32x16 acc[2][C::NTB];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < C::NTB; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[r][j][q] = 0.f;

    // this split's share of the K-blocks, by cost: a dense block one unit, a 2:4 block two
    const int units = a.nkb_d + 2 * a.nkb_s;
    const int u0 = (int)((int64_t)split * units / splits), u1 = (int)((int64_t)(split + 1) * units / splits);
    const int d0 = min(u0, a.nkb_d), d1 = min(u1, a.nkb_d);
    const int k0 = (max(u0, a.nkb_d) - a.nkb_d) / 2, k1 = split + 1 == splits ? a.nkb_s : (max(u1, a.nkb_d) - a.nkb_d) / 2;
    // tiles, and the token blocks that the XCDs work on at one time, start their loops at different blocks, so
    // that they do not all read the same rows of X or the same values at once
    auto turn = [&](int n) { return n > 0 ? (int)(((int64_t)t * n / a.n_tiles + (int64_t)((3 * tb) & 7) * n / 8) % n) : 0; };
    auto regions = [&](auto last) {
      constexpr bool LAST = decltype(last)::value;
      prefill_region<MX4, NT, true, LAST>(a, xs_a, xs_b, as_a, as_b, ms_a, ms_b, rx, rvd, rsd, rm, rid, t * a.nkb_d + d0,
                                          d1 - d0, turn(d1 - d0), rb, n0, hi, xlast, acc);
      prefill_region<MX4, NT, false, LAST>(a, xs_a, xs_b, as_a, as_b, ms_a, ms_b, rx, rvs, rss, rm, ris,
                                           t * a.nkb_s + k0, k1 - k0, turn(k1 - k0), rb, n0, hi, xlast, acc);
    };
    if (touch) regions(std::true_type{});
    else regions(std::false_type{});
    __syncthreads();

    if (splits > 1) {
      float flat[2 * C::NTB * 16];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < C::NTB; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q) flat[(r * C::NTB + j) * 16 + q] = acc[r][j][q];
      if (!join_splits(flat, part, counters, item, split, splits, &s_last)) continue;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < C::NTB; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q) acc[r][j][q] = flat[(r * C::NTB + j) * 16 + q];
    }

    // Y through LDS, 32 rows at a time: acc[r][j][q] is row m = 8 (q / 4) + 4 (lane / 32) + q % 4 of tile r, token tok_w + 32 j + lane % 32
    uint16_t* const ya = reinterpret_cast<uint16_t*>(xs_a);
    uint16_t* const yb = reinterpret_cast<uint16_t*>(xs_b);
    constexpr int PITCH = NT + 8;
    static_assert(32 * PITCH * 2 <= C::TILE, "32 rows of Y fit a tile");
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < C::NTB; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          (r ? yb : ya)[(8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)) * PITCH + tok_w + 32 * j + (lane & 31)] = to_bf16(acc[r][j][q]);
    __syncthreads();
    // 16-byte stores at 16-byte aligned addresses whatever the row's alignment: piece 0 of a row is what precedes
    // its first aligned address (unaligned stores made 11008 rows of 2047 tokens 14 us slower)
    for (int c = threadIdx.x; c < 64 * (C::CPR + 1); c += 256) {
      const int rr = c / (C::CPR + 1), k = c % (C::CPR + 1), m = rr & 31;
      uint16_t* dst = a.y + ((int64_t)t * a.rows + rb * 64 + rr) * a.ldy + n0;
      const int head = (int)(-(uintptr_t)dst / 2 % 8);
      const int at = k == 0 ? 0 : head + 8 * (k - 1), end = min(k == 0 ? head : at + 8, min(hi - n0, NT));
      const uint16_t* src = ((rr >> 5) ? yb : ya) + m * PITCH;
      if (end - at == 8 && at % 8 == 0) {
        *reinterpret_cast<u32x4*>(dst + at) = *reinterpret_cast<const u32x4*>(src + at);
      } else if (end - at == 8) {
        u32x4 v;
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = (uint32_t)src[at + 2 * u] | ((uint32_t)src[at + 2 * u + 1] << 16);
        *reinterpret_cast<u32x4*>(dst + at) = v;
      } else {
        for (int q = at; q < end; ++q) dst[q] = src[q];
      }
    }
    __syncthreads();                           // the tiles are the next item's
  }
}

// X rows into the workspace at a 16-byte aligned pitch, zeros behind them.
__global__ __launch_bounds__(256) void align_kernel(const uint16_t* __restrict__ x, int64_t ldx, int n_cols,
                                                    uint16_t* __restrict__ out, int64_t ld, int rows) {
  for (int r = blockIdx.y; r < rows; r += gridDim.y)
    for (int64_t n = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8; n < ld; n += (int64_t)gridDim.x * 2048) {
      const uint16_t* src = x + r * ldx + n;
      u32x4 v = {0u, 0u, 0u, 0u};
      if (n + 8 <= n_cols) v = *reinterpret_cast<const any_u32x4*>(src);
      else
        for (int u = 0; u < 8 && n + u < n_cols; ++u) v[u >> 1] |= (uint32_t)src[u] << (16 * (u & 1));
      *reinterpret_cast<u32x4*>(out + r * ld + n) = v;
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

// Tokens a workgroup takes, from the columns an expert has on average (the
// counts themselves are on the device): 16 or 32 in the decode kernel, 128 or
// 256 in the prefill kernel.  The decode kernel is the better one for few
// columns, and for more of them while it has no more than 768 items, three a
// compute unit of the four it runs at once (us, decode 32 against prefill 128,
// 4-bit: 11008x4096 at 128 tokens, 688 items, 18 against 23; at 200, 1204
// items, 30 against 28; 8 experts of 4096x4096, 39 columns on average, 21
// against 32; 55, 30 against 32).  Of the prefill's blocks, 256 halves the
// bytes of packed values, but costs an expert with few columns the whole
// block, and one a little above 256 two.  How many experts that is depends on
// the counts, which the average does not tell, so the steps for several
// experts are those of one weight and moderate skew, 8 experts of 4096x4096
// at top 2 (128 against 256, bf16, three routings each: 65 columns 30 against
// 42, 71 48 against 41, 87 46 against 41, 142 52 against 62, 172 53 against
// 41-64, 206 54-72 against 65, 237 72 against 65).  16 experts of 2048x4096
// follow them less well (71 49 against 39, 107 49 against 63) and 8 of
// 11008x4096 not below 172 columns, where 128 is the better one throughout (65
// 75-90 against 102, 107 93-115 against 107-122, 142 112-121 against 125).
// One weight of 11008x4096: 200 tokens 28 against 32, 400 44 against 40; of
// 2048x2048: 2048 tokens 19 against 29.
int token_block(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols) {
  const int64_t avg = (n_cols + n_experts - 1) / n_experts;
  if (avg <= (n_experts == 1 ? 16 : 20)) return 16;
  const int64_t some = n_experts > 1 ? std::min<int64_t>(n_experts, n_cols) / 4 : 0;   // blocks that are not full
  if ((n_experts > 1 && avg <= 48) || (p.cout / 64) * ((n_cols + 31) / 32 + some) <= 3 * kCus) return 32;
  if (n_experts == 1) return (p.cout / 64) * ((n_cols + 255) / 256) <= kCus ? 128 : 256;
  return avg <= 64 || (avg > 110 && avg <= 170) ? 128 : 256;
}

// Workspace: arrival counters and the partial sums of at most kMaxWgs
// workgroups, where a launch may split: with several experts when one token
// block would leave workgroups idle, with one expert when all columns would.
// A lone range shorter than the columns may leave them idle all the same; it
// then runs unsplit (may_split), so that what the product needs and its bits
// depend on what the host knows.  Behind them, for the kernel of many
// tokens and rows that are not 16-byte aligned, a copy of X with aligned rows:
// gathering unaligned rows made the 11008x4096 product over 2047 tokens 171 us
// where aligned ones take 111, and the copy takes 10.  The counters' place is
// kept free also where nothing splits: the next call with the same workspace
// may split, and counts on zeros there.
struct Workspace {
  int64_t split, copy, ld;           // bytes of counters and sums, bytes of the copy, the copy's row pitch (elements)
  int64_t copy_at() const { return std::max(split, hinm::kWsCounterBytes); }
  int64_t bytes() const { return copy ? copy_at() + copy : split; }
};
Workspace workspace_of(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols, bool x_aligned) {
  Workspace w{0, 0, 0};
  if (n_cols == 0) return w;
  const int nt = token_block(p, n_experts, n_cols);
  const int64_t fewest = (p.cout / 64) * (n_experts == 1 ? (n_cols + nt - 1) / nt : 1);   // items, if any
  if (fewest * 2 <= (nt <= 32 ? kCus : kMaxWgs)) w.split = hinm::kWsCounterBytes + (int64_t)kMaxWgs * nt * 64 * 4;
  if (nt >= 128 && !x_aligned) {
    w.ld = (n_cols + 7) / 8 * 8;
    w.copy = (p.cin * w.ld * 2 + 255) / 256 * 256;
  }
  return w;
}

// The product behind every entry point; `a` holds the weights' pointers.
template <bool MX4>
int launch(const hinm_plan_t& p, int32_t n_experts, ExpArgs a, const void* x, int64_t n_cols, int64_t ldx,
           const int32_t* starts, const int32_t* counts, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
           void* stream_) {
  const bool x_aligned = hinm::aligned(x, 16) && ldx % 8 == 0;
  const Workspace w = workspace_of(p, n_experts, n_cols, x_aligned);
  const int64_t need = w.bytes();
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
  a.may_split = w.split > 0;
  a.cin = p.cin;
  a.cout = p.cout;
  a.rows = p.tile_rows;
  a.n_tiles = p.n_tiles;
  a.nkb_d = p.n_dense_pad / HINM_KB_DENSE;
  a.nkb_s = p.n_24_pad / HINM_KB_24;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  a.x_end = 1;
  if (w.copy) {
    uint16_t* copy = reinterpret_cast<uint16_t*>(static_cast<char*>(workspace) + w.copy_at());
    const dim3 grid((unsigned)((w.ld + 2047) / 2048), (unsigned)std::min(p.cin, 4096));
    hipLaunchKernelGGL(align_kernel, grid, dim3(256), 0, stream, a.x, ldx, a.n_cols, copy, w.ld, p.cin);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return fail(HINM_EHIP, "experts launch: %s", hipGetErrorString(e));
    a.x = copy;
    a.ldx = ldx = w.ld;
    a.x_end = w.ld == n_cols;            // a multiple of 8 columns leaves the copy's rows no pad
  }
  // The fast kernels address X with 32-bit buffer offsets and 24-bit
  // multiplies (row number, row pitch in bytes).
  const int64_t x_bytes = ((int64_t)(p.cin - 1) * ldx + n_cols) * 2;
  if (x_bytes >= ((int64_t)1 << 31) - 16 || ldx * 2 >= (1 << 24) || p.cin > (1 << 24)) {
    const int64_t tbs = n_cols / kGenTok + std::min<int64_t>(n_experts, n_cols);
    const dim3 grid((unsigned)(p.cout / 64), (unsigned)std::min<int64_t>(tbs, 65535));
    hipLaunchKernelGGL(experts_general_kernel<MX4>, grid, dim3(256), 0, stream, a);
  } else {
    unsigned* ctr = static_cast<unsigned*>(workspace);
    float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + (w.split ? hinm::kWsCounterBytes : 0));
    const dim3 grid(kMaxWgs), block(256);
    switch (token_block(p, n_experts, n_cols)) {
      case 16: hipLaunchKernelGGL((experts_decode_kernel<MX4, 16>), dim3(kCus * decode_wgs(16)), block, 0, stream, a, part, ctr); break;
      case 32: hipLaunchKernelGGL((experts_decode_kernel<MX4, 32>), dim3(kCus * decode_wgs(32)), block, 0, stream, a, part, ctr); break;
      case 128: hipLaunchKernelGGL((experts_prefill_kernel<MX4, 128>), grid, block, 0, stream, a, part, ctr); break;
      default: hipLaunchKernelGGL((experts_prefill_kernel<MX4, 256>), grid, block, 0, stream, a, part, ctr); break;
    }
  }
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
                                                 int32_t x_aligned, size_t* bytes) {
  hinm::clear_error();
  int st = hinm::check_plan(plan);
  if (st) return st;
  st = check_args(*plan, n_experts, nullptr, 0, 0, nullptr, 0);
  if (st) return st;
  if (!bytes) return fail(HINM_EINVAL, "bytes is NULL");
  st = check_cols(n_cols);
  if (st) return st;
  const Workspace w = workspace_of(*plan, n_experts, n_cols, x_aligned != 0);
  *bytes = (size_t)w.bytes();
  return HINM_OK;
}

extern "C" int hinm_spmm_mx4_workspace_bytes(const hinm_plan_t* plan, int64_t batch, int32_t x_aligned,
                                             size_t* bytes) {
  return hinm_spmm_experts_workspace_bytes(plan, 1, batch, x_aligned, bytes);
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
