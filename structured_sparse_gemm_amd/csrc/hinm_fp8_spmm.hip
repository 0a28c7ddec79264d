// hinm_spmm_fp8, hinm_spmm_experts_fp8: products of packed weights with 8-bit
// values and activations rounded to 8 bits token by token (layout and formulas
// at hinm_fp8_t).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "hinm_device.h"
#include "hinm_fp8.h"
#include "hinm_internal.h"
#include "hinm_ragged.h"
#include "hinm_stream.h"

using hinm::Buf;
using hinm::check_bufs;
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

// The weights of all experts and a window of the activations' columns: x, y
// and n_cols are the window's, `before` columns precede it of `total`.  Strides
// are per expert.
struct Fp8Args {
  const uint8_t *val_d, *val_s, *scale_d, *scale_s, *meta, *idx_d, *idx_s;
  int64_t b_val_d, b_val_s, b_scale_d, b_scale_s, b_meta, b_idx_d, b_idx_s;   // bytes of one expert
  const uint16_t* x;                 // bf16 [cin][ldx]
  int64_t ldx;
  const uint8_t *x8, *xs;            // E4M3 [cin][ld8], E8M0 [ld8]
  int ld8;
  uint16_t* y;
  int64_t ldy;
  const int32_t *starts, *counts;    // NULL: one range, all columns
  int n_experts, n_cols, before, total;
  int may_split;                     // the workspace has room for partial sums
  int cin, cout, rows, n_tiles, nkb_d, nkb_s;
};

// Columns [lo, hi) of expert e within the window.
__device__ inline void range_of(const Fp8Args& a, int e, int& lo, int& hi) {
  lo = 0;
  hi = a.n_cols;
  if (!a.starts) return;
  const int s = a.starts[e], c = a.counts[e];
  if (s < 0 || c <= 0 || s >= a.total) {
    hi = 0;
    return;
  }
  lo = min(max(s - a.before, 0), a.n_cols);
  hi = min(max(s + min(c, a.total - s) - a.before, lo), a.n_cols);
}

// ---------------------------------------------------------------------------
// Activations to 8 bits.  The scale of a token needs its whole column, so one
// kernel takes the largest magnitudes of kChunks pieces of the channels and a
// second one combines them and rounds; the second read of X comes from the
// last-level cache.
// ---------------------------------------------------------------------------
constexpr int kChunks = 64;          // pieces of the channels

// Two bf16 magnitudes held as signed 16-bit numbers, 0x80 above their bits: what
// is not finite is negative then and loses to every other.
constexpr uint32_t kLeast = 0x00800080u;
typedef short i16x2 __attribute__((ext_vector_type(2)));
__device__ inline uint32_t larger2(uint32_t m, uint32_t v) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(i16x2, m), __builtin_bit_cast(i16x2, v)));
}
__device__ inline uint32_t larger(uint32_t m, uint32_t v) {        // v: two bf16 values
  return larger2(m, (v & 0x7fff7fffu) + kLeast);                   // no carry between the halves
}
template <int CTRL>
__device__ inline uint32_t moved(uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp((int)kLeast, (int)v, CTRL, 0xf, 0xf, false); }

// A token's scale byte from the largest magnitude as held above.
__device__ inline uint32_t column_scale(uint32_t held) { return fp8_scale_of(held - 0x80u); }

// Whether a token, or one of two, has values past 448 * 2^119, the largest
// code at the largest scale (at 2^120 the codes of bf16's largest values would
// stand for 2^128, which bf16 does not have); and two values saturated there,
// what is not finite left as it is.  The largest magnitudes are known where the
// scales are, so that only such tokens pay for it.
constexpr uint32_t kMostHeld = 0x7f60u + 0x80u;
__device__ inline bool far2(uint32_t held) { return (held & 0xffffu) > kMostHeld || held >> 16 > kMostHeld; }
__device__ inline uint32_t saturated(uint32_t v) {
  const uint32_t lo = v & 0x7fffu, hi = v & 0x7fff0000u;
  if (lo > 0x7f60u && lo < 0x7f80u) v = (v & 0xffff8000u) | 0x7f60u;
  if (hi > 0x7f600000u && hi < 0x7f800000u) v = (v & 0x8000ffffu) | 0x7f600000u;
  return v;
}
__device__ inline u32x4 saturated(u32x4 v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = saturated(v[k]);
  return v;
}
template <int N>
__device__ inline void saturate(u32x4 (&v)[N]) {
#pragma unroll
  for (int u = 0; u < N; ++u) v[u] = saturated(v[u]);
}

// Eight values as codes; the conversion makes NaN of what is not finite.
__device__ inline fp8_u32x2 column_codes(u32x4 v, const float (&inv)[8]) {
  fp8_u32x2 c = {0u, 0u};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float lo = __uint_as_float(v[k] << 16) * inv[2 * k], hi = __uint_as_float(v[k] & 0xffff0000u) * inv[2 * k + 1];
    c[k >> 1] = (k & 1) ? (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, (int)c[k >> 1], true)
                        : (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(lo, hi, (int)c[k >> 1], false);
  }
  return c;
}

// Workgroup: 256 columns (32 threads of 8), 8 rows at a time of one piece, whose
// rows (up to 8 a thread) are all in flight at once: four at a time, and loads
// under a condition, took 25 and 23 us for 11008 x 2047 values, this 11 and 17,
// 4.2 and 4.0 TB/s.  A thread's columns are the window's last eight where it has
// no eight more, so that two threads may write the same values; a window of
// fewer than eight columns is read one by one.
constexpr int kRowsHeld = 8;
__device__ __forceinline__ void load_rows(const Fp8Args& a, int n, int r0, int r1, u32x4 (&v)[kRowsHeld]) {
  const int first = r0 + (threadIdx.x >> 5);
#pragma unroll
  for (int u = 0; u < kRowsHeld; ++u) {
    const uint16_t* const row = a.x + (int64_t)min(first + 8 * u, r1 - 1) * a.ldx + n;
    if (a.n_cols >= 8) {
      v[u] = *reinterpret_cast<const any_u32x4*>(row);
    } else {
      v[u] = u32x4{0u, 0u, 0u, 0u};
      for (int k = 0; k < a.n_cols; ++k) v[u][k >> 1] |= (uint32_t)row[k] << (16 * (k & 1));
    }
  }
}

__global__ __launch_bounds__(256) void fp8_colmax_kernel(Fp8Args a, uint16_t* __restrict__ part) {
  __shared__ u32x4 sh[256];
  const int r0 = (int)((int64_t)blockIdx.y * a.cin / gridDim.y), r1 = (int)((int64_t)(blockIdx.y + 1) * a.cin / gridDim.y);
  const int n = max(min((int)(blockIdx.x * 256 + 8 * (threadIdx.x & 31)), a.n_cols - 8), 0);
  u32x4 m = {kLeast, kLeast, kLeast, kLeast};
  for (int r = r0; r < r1; r += 8 * kRowsHeld) {
    u32x4 v[kRowsHeld];
    load_rows(a, n, r, r1, v);
#pragma unroll
    for (int u = 0; u < kRowsHeld; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = larger(m[k], v[u][k]);
  }
  sh[threadIdx.x] = m;
  __syncthreads();
  if (threadIdx.x < 32) {
    for (int k = 1; k < 8; ++k)
#pragma unroll
      for (int u = 0; u < 4; ++u) m[u] = larger2(m[u], sh[32 * k + threadIdx.x][u]);
    *reinterpret_cast<any_u32x4*>(part + (int64_t)blockIdx.y * a.ld8 + n) = m;
  }
}

__global__ __launch_bounds__(256) void fp8_columns_kernel(Fp8Args a, const uint16_t* __restrict__ part, int chunks,
                                                          uint8_t* __restrict__ x8, uint8_t* __restrict__ xs) {
  typedef fp8_u32x2 any_u32x2 __attribute__((aligned(1)));
  __shared__ u32x4 sh[256];
  const int r0 = (int)((int64_t)blockIdx.y * a.cin / gridDim.y), r1 = (int)((int64_t)(blockIdx.y + 1) * a.cin / gridDim.y);
  const int n = max(min((int)(blockIdx.x * 256 + 8 * (threadIdx.x & 31)), a.n_cols - 8), 0);
  u32x4 v[kRowsHeld], m = {kLeast, kLeast, kLeast, kLeast};
  load_rows(a, n, r0, r1, v);
#pragma unroll 8
  for (int k = threadIdx.x >> 5; k < chunks; k += 8) {
    const u32x4 t = *reinterpret_cast<const any_u32x4*>(part + (int64_t)k * a.ld8 + n);
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = larger2(m[u], t[u]);
  }
  sh[threadIdx.x] = m;
  __syncthreads();
  for (int k = 0; k < 8; ++k)
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = larger2(m[u], sh[32 * k + (threadIdx.x & 31)][u]);
  uint32_t e[8];
  float inv[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    e[u] = column_scale((m[u >> 1] >> (16 * (u & 1))) & 0xffffu);
    inv[u] = fp8_inverse(e[u]);
  }
  const bool far = far2(m[0]) || far2(m[1]) || far2(m[2]) || far2(m[3]);
  if (blockIdx.y == 0 && threadIdx.x < 32)
    for (int u = 0; u < 8; ++u) xs[n + u] = (uint8_t)e[u];
  for (int r = r0;;) {
#pragma unroll
    for (int u = 0; u < kRowsHeld; ++u) {
      const int row = r + (threadIdx.x >> 5) + 8 * u;
      if (far) v[u] = saturated(v[u]);
      if (row < r1) *reinterpret_cast<any_u32x2*>(x8 + (int64_t)row * a.ld8 + n) = column_codes(v[u], inv);
    }
    if ((r += 8 * kRowsHeld) >= r1) break;
    load_rows(a, n, r, r1, v);
  }
}

// ---------------------------------------------------------------------------
// Many tokens.  Workgroup = 64 rows x NT tokens, four waves of 64 rows x NT / 4
// tokens.  Everything goes straight from memory into LDS: the gathered X rows
// two blocks ahead into a ring of three tiles, the weight's blocks (values,
// metadata, scales, indices) four blocks ahead into a ring of five slots, so
// that the indices of a block's rows have come when its rows are asked for.
// Codes of both sides become bf16 between LDS and the matrix instruction.
//
// A wave's loads complete in order, and at the end of step b those of step
// b - 1 must have: what step b asked for has two steps' time.  The weight's
// blocks need it: they come from the last-level cache or from memory, some two
// thousand cycles away (with __syncthreads(), which waits for all loads into
// LDS, 4096x11008 at 2047 tokens took 87 us, and 67 without the rows or without
// the products).  Hence the loads are inline assembly, which the compiler does
// not wait for, and the barrier waits for LDS operations alone.  What a step
// issues beside its 48 conversions and 8 products bounds it next: with the
// addresses of the weight's blocks worked out anew in every step, and one loop
// for both kinds of blocks, 96 us, with addresses that move on 79 (587 TFLOP/s
// of kept products).
//
// Tile layout: position p's row of NT bytes, its 16-byte chunk c at chunk
// c ^ turned(p), so that a 32-lane half of a transposed read covers every bank
// once.  An expert's token blocks start at multiples of 16 columns (aligned
// loads of codes); columns before its first are not written.
// ---------------------------------------------------------------------------
template <int NT>
struct Pre {
  static constexpr int TW = NT / 4;            // tokens of a wave
  static constexpr int NTB = TW / 32;          // 32-token tiles of a wave
  static constexpr int CPR = NT / 16;          // 16-byte chunks of a row
  static constexpr int RPL = 64 / CPR;         // positions of one load
  static constexpr int TILE = 64 * NT;         // bytes of an X tile
};
template <int NT>
__device__ inline int turned(int p) { return NT == 256 ? 2 * (p & 7) : 2 * ((p >> 1) & 3); }

// A slot of the weight's ring: 64 rows' values of a block, then what one load
// brings: metadata, scales and indices.
constexpr int kTiles = 3, kRing = 5, kMeta = 2048, kScale = kMeta + 512, kIndex = kScale + 64, kSlot = kMeta + 1024;

// Sixteen bytes a lane into LDS at `lds` + 16 lane: from a buffer (past its end
// zeros; sc0 as in load_lds16), and from an address.
__device__ inline void lds_load(u32x4 buffer, uint32_t lds, uint32_t offset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen sc0 lds"
               :: "s"(lds), "v"(offset), "s"(buffer) : "m0", "memory");
}
__device__ inline void lds_load(const uint8_t* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" :: "s"(lds), "v"(src) : "m0", "memory");
}

// An item: row block rb of tile t of an expert, blocks d0 .. d0 + nd - 1 of its
// dense region and k0 .. k0 + ns - 1 of its 2:4 region, each region from its
// block turn on and around; the dense ones first.
struct Work {
  const uint8_t *val_d, *val_s, *scale_d, *scale_s, *meta, *idx_d, *idx_s;
  int tile, rb, d0, nd, turn_d, k0, ns, turn_s;
};

template <int NT>
__device__ __forceinline__ void multiply_weight(const Fp8Args& a, const Work w, uint8_t* lds, u32x4 rx, int n0,
                                                const float (&xs)[Pre<NT>::NTB], f32x16 (&acc)[2][Pre<NT>::NTB]) {
  using C = Pre<NT>;
  constexpr int NJ = 16 / C::RPL;              // X loads of a wave for 64 positions
  const int lane = threadIdx.x & 63, nb = w.nd + w.ns;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint8_t* const ring = lds + kTiles * C::TILE;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)lds, ring0 = lds0 + kTiles * C::TILE;
  // offsets in the rings move on by a step
  auto next_tile = [](uint32_t& t) { t = t == (kTiles - 1) * C::TILE ? 0u : t + C::TILE; };
  auto next_slot = [](uint32_t& t) { t = t == (kRing - 1) * kSlot ? 0u : t + kSlot; };

  // The weight's blocks in the order of the loop, into a slot each: waves 0 and 1 (and 3 again) half of the values each,
  // wave 2 in lanes 0 .. 31 metadata (a dense block has none and reads values), 32 .. 35 scales, the others indices, the
  // last sixteen bytes again where there are no more.  A lane's address moves on by its stride; up to four runs of
  // adjacent blocks, two a region, begin anew.  Past the end the last block is read again: waits are for known numbers
  // of loads.
  const uint32_t into = ring0 + (wave == 2 ? kMeta : 1024u * (wave == 1));
  const uint8_t* src = nullptr;
  uint32_t stride = 0, stride4 = 0;            // stride4: from the last block of four that share scales
  uint32_t slot_w = 0;
  int run = -1, left = 0, kw = 0;              // of the run; the block's number in its region
  auto begin_run = [&] {
    int first = 0;
    do {
      ++run;
      const int n = run < 2 ? w.nd : w.ns, turn = run < 2 ? w.turn_d : w.turn_s;
      first = (run & 1) ? 0 : turn;
      left = (run & 1) ? turn : n - turn;
    } while (left == 0);                       // some run follows: a block is left
    const bool dense = run < 2;
    kw = (dense ? w.d0 : w.k0) + first;
    const int nkb = dense ? a.nkb_d : a.nkb_s;
    const int64_t kb = (int64_t)w.tile * nkb + kw, row = kb * a.rows + w.rb * 64;
    src = (dense ? w.val_d : w.val_s) + row * 32 + 1024 * (wave == 1) + 16 * lane;
    stride = stride4 = a.rows * 32;
    if (wave == 2) {
      if (!dense) src = w.meta + row * 8 + 16 * lane, stride = stride4 = a.rows * 8;
      if (lane >= 36) {
        src = (dense ? w.idx_d : w.idx_s) + kb * (dense ? 128 : 256) + 16 * min(lane - 36, dense ? 7 : 15);
        stride = stride4 = dense ? 128 : 256;
      } else if (lane >= 32) {
        src = (dense ? w.scale_d : w.scale_s) + ((int64_t)w.tile * ((nkb + 3) / 4) + kw / 4) * a.rows + w.rb * 64 + 16 * (lane - 32);
        stride = 0;
        stride4 = a.rows;
      }
    }
  };
  int blocks = nb;                             // not asked for yet
  auto load_weight = [&] {
    if (blocks > 0) {
      if (left == 0) {
        begin_run();
      } else {
        src += (kw & 3) == 3 ? stride4 : stride;
        ++kw;
      }
      --left;
      --blocks;
    }
    lds_load(src, into + slot_w);
    next_slot(slot_w);
  };
  // A wave stages 16 positions of a 2:4 block, or 8 of a dense one, RPL a load: load j those from first + RPL j on,
  // first a multiple of 8 or 16, so that turned() is the same for both.
  const int q = lane / C::CPR, sl = lane % C::CPR;
  uint32_t xoff[NJ];                           // source byte in a row; past the buffer for columns past its rows
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int n = n0 + 16 * (sl ^ turned<NT>(j * C::RPL + q));
    xoff[j] = n < a.ld8 ? (uint32_t)n : 0x80000000u;
  }
  uint32_t tile_x = 0, slot_x = 0;
  auto load_x = [&](int b) {
    auto rows = [&](auto count, int first) {
      const int* index = reinterpret_cast<const int*>(ring + slot_x + kIndex) + first + q;
      int c[decltype(count)::value];
#pragma unroll
      for (int j = 0; j < decltype(count)::value; ++j) c[j] = index[j * C::RPL];
#pragma unroll
      for (int j = 0; j < decltype(count)::value; ++j)       // both factors are below 2^24
        lds_load(rx, lds0 + tile_x + (first + j * C::RPL) * NT,
                 (uint32_t)c[j] < (uint32_t)a.cin ? __umul24((uint32_t)c[j], (uint32_t)a.ld8) + xoff[j] : kOob);
    };
    if (b < w.nd) rows(std::integral_constant<int, NJ / 2>{}, wave * 8);
    else rows(std::integral_constant<int, NJ>{}, wave * 16);
    next_tile(tile_x);
    if (b < nb - 1) next_slot(slot_x);         // past the end the last block's rows again
  };
  // until all but block b's rows and `more` other loads have come
  auto wait_but = [&](int b, auto more) {
    if (b < w.nd) wait_vm<NJ / 2 + decltype(more)::value>();
    else wait_vm<NJ + decltype(more)::value>();
  };
  const int m32 = lane & 31, h = lane >> 5;    // operand row or column, and half of the positions
  const int tg = (lane >> 4) & 1, p = (lane & 15) >> 1, s8 = lane & 1;
  // The lane's share of a transposed read: the row of its position in the first
  // read of instruction 0.  Instruction s's positions are 16 s + 8 h + p, and 32
  // further on.  A dense block is multiplied as a 2:4 block whose groups keep
  // positions 0 and 1 - column 2 q + u at 4 q + u, as many instructions as the
  // dense ones would be - and positions 4 q + 2, + 3, which nothing reads, take
  // those rows again.
  const int row24 = 8 * h + p, row_dense = 4 * h + 2 * (p >> 2) + (p & 1);
  uint32_t off24[C::NTB], off_dense[C::NTB];
#pragma unroll
  for (int j = 0; j < C::NTB; ++j) {
    const int chunk = wave * (C::TW / 16) + 2 * j + tg;
    off24[j] = (uint32_t)(row24 * NT + 16 * (chunk ^ turned<NT>(row24)) + 8 * s8);
    off_dense[j] = (uint32_t)(row_dense * NT + 16 * (chunk ^ turned<NT>(row_dense)) + 8 * s8);
  }
  uint32_t tile_c = 0, slot_c = 0;
  // Half h of instruction s takes the row's values 8 (2 h + s) .. + 7, so that a
  // lane's values of both instructions are 16 adjacent bytes.
  auto compute = [&](auto dense_block) {
    constexpr bool dense = decltype(dense_block)::value;
    constexpr int second = dense ? 8 * NT : 16 * NT;
    const uint8_t *xt = lds + tile_c, *slot = ring + slot_c;
    // all of the block's LDS reads first: with two waves a SIMD little else hides their latency
    float scale[2];
    u32x4 v[2];
    uint32_t m[2];
    fp8_u32x2 raw[2][C::NTB][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      scale[r] = fp8_scale(slot[kScale + 32 * r + m32]);
      v[r] = *reinterpret_cast<const u32x4*>(slot + (32 * r + m32) * 32 + 16 * h);
      m[r] = dense ? 0x44444444u : *reinterpret_cast<const uint32_t*>(slot + kMeta + (32 * r + m32) * 8 + 4 * h);
    }
#pragma unroll
    for (int j = 0; j < C::NTB; ++j) {
      const uint8_t* const at = xt + (dense ? off_dense[j] : off24[j]);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int u = 0; u < 2; ++u) raw[s][j][u] = tr_read8(at + (s + 2 * u) * second);
    }
    __builtin_amdgcn_sched_barrier(0);
    bf16x8 av[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      av[r][0] = __builtin_bit_cast(bf16x8, fp8_expand(fp8_u32x2{v[r][0], v[r][1]}, scale[r]));
      av[r][1] = __builtin_bit_cast(bf16x8, fp8_expand(fp8_u32x2{v[r][2], v[r][3]}, scale[r]));
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < C::NTB; ++j) {
        const bf16x8 lo8 = __builtin_bit_cast(bf16x8, fp8_expand(raw[s][j][0], xs[j]));
        const bf16x8 hi8 = __builtin_bit_cast(bf16x8, fp8_expand(raw[s][j][1], xs[j]));
        const bf16x16 bv = __builtin_shufflevector(lo8, hi8, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
        for (int r = 0; r < 2; ++r)
          acc[r][j] = __builtin_amdgcn_smfmac_f32_32x32x32_bf16(av[r][s], bv, acc[r][j], (int)(s ? m[r] >> 16 : m[r]), 0, 0);
      }
    next_tile(tile_c);
    next_slot(slot_c);
  };
  auto step = [&](int b, auto dense_block) {
    __builtin_amdgcn_s_setprio(2);             // the loads go out ahead of the other workgroup's arithmetic
    load_x(b + 2);
    load_weight();
    __builtin_amdgcn_s_setprio(0);
    compute(dense_block);
    wait_but(b + 2, std::integral_constant<int, 1>{});
    step_barrier();
  };

  step_barrier();                              // LDS is free
  wait_vm<0>();                                // counted loads begin here
  for (int b = 0; b < kRing - 1; ++b) load_weight();
  wait_vm<kRing - 3>();                        // the indices of blocks 0 and 1
  step_barrier();
  load_x(0);
  load_x(1);
  wait_but(1, std::integral_constant<int, 0>{});
  step_barrier();
  int b = 0;
#pragma nounroll
  for (; b < w.nd; ++b) step(b, std::true_type{});
#pragma nounroll
  for (; b < nb; ++b) step(b, std::false_type{});
  wait_vm<0>();                                // what was loaded past the end
}

constexpr int kPreThreads = 256;

template <int NT>
__global__ __launch_bounds__(kPreThreads, 2) void fp8_prefill_kernel(Fp8Args a, float* __restrict__ part,
                                                                     unsigned* __restrict__ counters) {
  using C = Pre<NT>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kTiles * C::TILE + kRing * kSlot];
  __shared__ int pre[HINM_MAX_EXPERTS + 1];
  __shared__ int s_last;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nrb = a.rows / 64, n_rb = a.n_tiles * nrb;
  const int tok_w = wave * C::TW;

  const int items = plan_blocks(a, NT, pre, 16) * n_rb;
  int splits = 1;
  while (a.may_split && splits < 4 && items * splits * 2 <= (int)gridDim.x && a.nkb_d + 2 * a.nkb_s >= 16 * splits)
    splits *= 2;
  const int xcd = blockIdx.x % 8, slot = blockIdx.x / 8, per_xcd = gridDim.x / 8;
  const int w_lo = (int)((int64_t)xcd * items * splits / 8), w_hi = (int)((int64_t)(xcd + 1) * items * splits / 8);
  const uint64_t x8 = reinterpret_cast<uint64_t>(a.x8);
  const u32x4 rx = {(uint32_t)x8, (uint32_t)(x8 >> 32), (uint32_t)a.cin * (uint32_t)a.ld8, (uint32_t)kBufferWord3};

  for (int work = w_lo + slot; work < w_hi; work += per_xcd) {
    const int item = work / splits, split = work % splits;
    const int tb = item / n_rb, trb = item % n_rb, t = trb / nrb, rb = trb % nrb;
    const int e = find_expert(a, pre, tb);
    int lo, hi;
    range_of(a, e, lo, hi);
    const int n0 = (lo & -16) + (tb - (a.starts ? pre[e] : 0)) * NT;

    // this split's share of the K-blocks, by cost: a dense block one unit, a 2:4 block two
    const int units = a.nkb_d + 2 * a.nkb_s;
    const int u0 = (int)((int64_t)split * units / splits), u1 = (int)((int64_t)(split + 1) * units / splits);
    const int d0 = min(u0, a.nkb_d), d1 = min(u1, a.nkb_d);
    const int k0 = (max(u0, a.nkb_d) - a.nkb_d) / 2, k1 = split + 1 == splits ? a.nkb_s : (max(u1, a.nkb_d) - a.nkb_d) / 2;
    // tiles, and the token blocks that the XCDs work on at one time, start their loops at different blocks, so
    // that they do not all read the same rows of X or the same values at once
    auto turn = [&](int n) { return n > 0 ? (int)(((int64_t)t * n / a.n_tiles + (int64_t)((3 * tb) & 7) * n / 8) % n) : 0; };
    const Work w{a.val_d + e * a.b_val_d, a.val_s + e * a.b_val_s, a.scale_d + e * a.b_scale_d, a.scale_s + e * a.b_scale_s,
                 a.meta + e * a.b_meta, a.idx_d + e * a.b_idx_d, a.idx_s + e * a.b_idx_s,
                 t, rb, d0, d1 - d0, turn(d1 - d0), k0, k1 - k0, turn(k1 - k0)};
    f32x16 acc[2][C::NTB];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < C::NTB; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[r][j][q] = 0.f;
    if (w.nd + w.ns > 0) {
      float xs[C::NTB];                            // scales of this lane's tokens
#pragma unroll
      for (int j = 0; j < C::NTB; ++j) xs[j] = fp8_scale(a.xs[min(n0 + tok_w + 32 * j + (lane & 31), a.ld8 - 1)]);
      multiply_weight<NT>(a, w, lds, rx, n0, xs, acc);
    }
    __syncthreads();

    if (splits > 1) {
      float flat[2 * C::NTB * 16];
#pragma unroll
      for (int k = 0; k < 2 * C::NTB * 16; ++k) flat[k] = acc[k / (16 * C::NTB)][k / 16 % C::NTB][k % 16];
      if (!join_splits(flat, part, counters, item, split, splits, &s_last)) continue;
#pragma unroll
      for (int k = 0; k < 2 * C::NTB * 16; ++k) acc[k / (16 * C::NTB)][k / 16 % C::NTB][k % 16] = flat[k];
    }

    // Y through LDS: acc[r][j][q] is row m = 8 (q / 4) + 4 (lane / 32) + q % 4 of half r,
    // token tok_w + 32 j + lane % 32
    uint16_t* const ys = reinterpret_cast<uint16_t*>(lds);
    static_assert(64 * NT * 2 <= kTiles * C::TILE, "64 rows of Y fit the tiles");
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int j = 0; j < C::NTB; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q)
          ys[(32 * r + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3)) * NT + tok_w + 32 * j + (lane & 31)] = to_bf16(acc[r][j][q]);
    __syncthreads();
    // 16-byte stores at 16-byte aligned addresses whatever the row's alignment: piece 0 of a row is what precedes its
    // first aligned address
    const int from = max(lo - n0, 0), to = min(hi - n0, NT);
    constexpr int PIECES = NT / 8 + 1;
    for (int c = threadIdx.x; c < 64 * PIECES; c += kPreThreads) {
      const int rr = c / PIECES, k = c % PIECES;
      uint16_t* dst = a.y + ((int64_t)t * a.rows + rb * 64 + rr) * a.ldy + n0;
      const int head = (int)(-(uintptr_t)dst / 2 % 8);
      const int at = max(k == 0 ? 0 : head + 8 * (k - 1), from), end = min(k == 0 ? head : head + 8 * k, to);
      const uint16_t* src = ys + rr * NT;
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

// ---------------------------------------------------------------------------
// Few tokens an expert: a read of the packed weight, one launch.  The codes of a
// segment's tokens (up to 16 of an expert) are held in LDS whole, [channel]
// [token], rounded there by every workgroup for itself; the transposed LDS read
// takes an address a lane, so the channels that a tile keeps are gathered there
// and every global load is at an address known beforehand.  An item is 16 F
// rows of a segment; a workgroup takes a contiguous range of items, its waves
// deal the K-blocks among themselves, and their sums meet in LDS.
// ---------------------------------------------------------------------------
constexpr int kDecThreads = 512, kDecWaves = kDecThreads / 64;
constexpr int kDecLds = 159360;      // bytes for the codes, a row of zeros and the waves' sums
constexpr int dec_red_bytes(int f) { return kDecWaves * (256 * f + 8) * 4; }   // the 8: reads free of bank conflicts
constexpr bool dec_fits(int64_t cin, int width, int f) { return (cin + 1) * width + dec_red_bytes(f) <= kDecLds; }

template <int F>
struct DecOperand {
  fp8_u32x2 v[F];
  uint32_t m[F], scale[F];
  int index;
};

struct DecSource {
  const uint8_t *val_d, *val_s, *meta, *idx_d, *idx_s, *scale_d, *scale_s;
  int tile, row, first, end;
};

// The activations of a segment: `width` columns, eight from n0 and, at width 16,
// eight from n1 on, of which columns lo .. hi - 1 are the segment's.
struct Segment {
  int n0, n1, lo, hi;
};

// X's values are kept in registers, kHeld loads a thread, from `load_x`, which
// comes ahead of the weight's first loads, to `round_x`: one pass of
// kHeld * 512 loads of sixteen bytes.  A load is eight columns of a channel -
// at width 16 neighbouring lanes take the two halves of a channel, which share
// cache lines - or, where X is one column without padding (TOKEN), eight
// channels.  Of fewer than eight columns a row's load reaches into the next
// rows, whose codes nothing uses, and the last rows' begins early and is shifted.
constexpr int kChannelLoads = 16;
template <bool TOKEN>
constexpr int kHeld = TOKEN ? (kDecLds / 8 + 8 * kDecThreads - 1) / (8 * kDecThreads) : kChannelLoads;
static_assert(kDecThreads == 512 && kChannelLoads == 16);          // the shifts below

template <bool TOKEN>
__device__ __forceinline__ void load_x(const Fp8Args& a, const Segment& sg, int width, int pass, u32x4 (&v)[kHeld<TOKEN>]) {
  const int tid = own_thread();
  if constexpr (TOKEN) {
#pragma unroll
    for (int u = 0; u < kHeld<TOKEN>; ++u) v[u] = *reinterpret_cast<const any_u32x4*>(a.x + min(8 * (tid + u * kDecThreads), a.cin - 8));
    return;
  }
  const int half = width == 16 ? tid & 1 : 0, shift = width == 16 ? 8 : 9, first = width == 16 ? tid >> 1 : tid;
  const int n0 = sg.n0, n1 = sg.n1;
  const uint16_t* const x = a.x + (half ? n1 : n0);
  const int64_t last = a.n_cols < 8 ? (int64_t)(a.cin - 1) * a.ldx + a.n_cols - 8 : INT64_MAX;
#pragma unroll
  for (int u = 0; u < kHeld<TOKEN>; ++u) {
    const int c = min(first + ((pass * kChannelLoads + u) << shift), a.cin - 1);
    v[u] = *reinterpret_cast<const any_u32x4*>(x + min((int64_t)((uint64_t)(uint32_t)c * (uint32_t)a.ldx), last));
  }
}

// Their codes into the slab, [channel][width] and a row of zeros, and the
// columns' scale bytes into `scales`.  Where one pass does not hold the columns,
// all but the last are read once more, from L2.
template <bool TOKEN>
__device__ __forceinline__ void round_x(const Fp8Args& a, const Segment& sg, int width, u32x4 (&v)[kHeld<TOKEN>], uint8_t* slab,
                                        uint32_t* red, uint8_t* scales) {
  const int tid = own_thread(), lane = tid & 63, passes = TOKEN ? 1 : (a.cin + (width == 16 ? 4095 : 8191)) >> (width == 16 ? 12 : 13);
  const int half = width == 16 ? tid & 1 : 0, shift = width == 16 ? 8 : 9, first = width == 16 ? tid >> 1 : tid;
  auto shift_last = [&](int pass) {
    if constexpr (TOKEN) {
#pragma unroll
      for (int u = 0; u < kHeld<TOKEN>; ++u) {
        const int c = 8 * (tid + u * kDecThreads);
        v[u] = shifted_row(v[u], min(max(c - (a.cin - 8), 0), 7));
      }
    } else if (a.n_cols < 8) {
      const int64_t last = (int64_t)(a.cin - 1) * a.ldx + a.n_cols - 8;
#pragma unroll
      for (int u = 0; u < kHeld<TOKEN>; ++u) {
        const int c = min(first + ((pass * kChannelLoads + u) << shift), a.cin - 1);
        v[u] = shifted_row(v[u], (int)max((int64_t)((uint64_t)(uint32_t)c * (uint32_t)a.ldx) - last, (int64_t)0));
      }
    }
  };
  u32x4 m = {kLeast, kLeast, kLeast, kLeast};
  shift_last(0);
#pragma nounroll
  for (int pass = 0;;) {
#pragma unroll
    for (int u = 0; u < kHeld<TOKEN>; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) m[k] = larger(m[k], v[u][k]);
    if (++pass == passes) break;
    load_x<TOKEN>(a, sg, width, pass, v);
    shift_last(pass);
  }
  // the largest of a wave's lanes (of equal parity at width 16), then of the waves: red[wave][half][4]
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t r = m[k];
    if (width == 8) r = larger2(r, moved<0x121>(r));
    r = larger2(r, moved<0x122>(r));
    r = larger2(r, moved<0x124>(r));
    r = larger2(r, moved<0x128>(r));
    r = larger2(r, (uint32_t)__shfl_xor((int)r, 16));
    m[k] = larger2(r, (uint32_t)__shfl_xor((int)r, 32));
  }
  if constexpr (TOKEN) {                                     // one column
    uint32_t t = larger2(larger2(m[0], m[1]), larger2(m[2], m[3]));
    t = larger2(t, t >> 16 | t << 16);
    m = u32x4{t, t, t, t};
  }
  if (lane < 2) *reinterpret_cast<u32x4*>(red + 8 * (tid >> 6) + 4 * lane) = m;
  step_barrier();
  uint32_t r = red[lane];
  r = larger2(r, moved<0x128>(r));
  r = larger2(r, (uint32_t)__shfl_xor((int)r, 16));
  r = larger2(r, (uint32_t)__shfl_xor((int)r, 32));
  const uint32_t e0 = column_scale(r & 0xffffu), e1 = column_scale(r >> 16);
  const bool far = __ballot(far2(r)) != 0;                   // of the whole segment
  if (tid < 8) *reinterpret_cast<uint16_t*>(scales + 2 * tid) = (uint16_t)(e0 | e1 << 8);
  const uint32_t i0 = __float_as_uint(fp8_inverse(e0)), i1 = __float_as_uint(fp8_inverse(e1));
  float inv[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const uint32_t from = u & 1 ? i1 : i0;
    const int lo = __builtin_amdgcn_readlane((int)from, u >> 1), hi = __builtin_amdgcn_readlane((int)from, 4 + (u >> 1));
    inv[u] = __int_as_float(half ? hi : lo);
  }
  if (tid < width / 8) *reinterpret_cast<fp8_u32x2*>(slab + a.cin * width + 8 * tid) = fp8_u32x2{0u, 0u};
  if constexpr (TOKEN) {
    if (far) saturate(v);
#pragma unroll
    for (int u = 0; u < kHeld<TOKEN>; ++u) {
      const int c = 8 * (tid + u * kDecThreads);
      if (c >= a.cin) break;
      const uint64_t code = __builtin_bit_cast(uint64_t, column_codes(v[u], inv));
      const int turn = tid >> 2;                   // lanes that share banks begin at other channels
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int j = (k + turn) & 7;
        if (c + j < a.cin) slab[(c + j) * 8] = (uint8_t)(code >> (8 * j));
      }
    }
    return;
  }
#pragma nounroll
  for (int pass = passes - 1;;) {
    if (far) saturate(v);
#pragma unroll
    for (int u = 0; u < kHeld<TOKEN>; ++u) {
      const int c = first + ((pass * kChannelLoads + u) << shift);
      if (c < a.cin) *reinterpret_cast<fp8_u32x2*>(slab + c * width + 8 * half) = column_codes(v[u], inv);
    }
    if (--pass < 0) break;
    load_x<TOKEN>(a, sg, width, pass, v);
    shift_last(pass);
  }
}

// Width: columns of a segment, 8 or 16.  Every instruction of the prologue is
// issued by every wave, and a compute unit's waves share its issue slots: of 4,
// 8 and 16 waves, 8 (16: a token 26 us).
template <int F, bool TOKEN>
__global__ __launch_bounds__(kDecThreads) void fp8_decode_kernel(Fp8Args a, int columns) {
  const int width = TOKEN ? 8 : columns;
  // 1, 2, 3 and 4: one token of 4096x11008 11.4, 10.0, 10.0 and 10.2 us, 8 experts of 11008x4096 with 8 columns 44.7,
  // 44.0, 51.2 and 47.9, 64 of 1408x2048 36, 37, 40 and 44 (three sets of inputs in turn)
  constexpr int kDepth = 2;
  __shared__ __attribute__((aligned(16))) uint8_t slab[kDecLds];
  __shared__ __attribute__((aligned(16))) uint32_t top[kDecWaves * 8];
  __shared__ int pre[HINM_MAX_EXPERTS + 1];
  __shared__ __attribute__((aligned(8))) uint8_t scales[16];
  float* const red = reinterpret_cast<float*>(slab + (kDecLds - dec_red_bytes(F)));
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63, i16 = lane & 15, kc = lane >> 4;
  const int nd = a.nkb_d, ns = a.nkb_s, nblk = nd + ns;
  const unsigned n_rb = a.cout / (16 * F);
  const Share mine = share_of(plan_blocks(a, width, pre), n_rb);
  int held = -1, coming = -1, rb = 0;
  Segment now{}, next{};
  u32x4 v[kHeld<TOKEN>];
  float xs = 1.f;
  f32x4 acc[F];
  stream<DecOperand<F>, DecSource, kDepth, kDecWaves>(
      (int)mine.n,
      [&](int i) -> DecSource {
        const unsigned sg = (mine.first + i) / n_rb, r16 = (mine.first + i - sg * n_rb) * F, t = r16 * 16 / (unsigned)a.rows;
        const int e = find_expert(a, pre, sg);
        if ((int)sg != coming) {
          coming = sg;
          range_of(a, e, next.lo, next.hi);
          next.lo += (sg - (a.starts ? pre[e] : 0)) * width;
          // eight columns each that X has, and of which some may be others'
          next.n0 = max(min(next.lo, a.n_cols - 8), 0);
          next.n1 = max(min(next.lo + 8, a.n_cols - 8), 0);
          load_x<TOKEN>(a, next, width, 0, v);
        }
        return {a.val_d + e * a.b_val_d, a.val_s + e * a.b_val_s, a.meta + e * a.b_meta, a.idx_d + e * a.b_idx_d,
                a.idx_s + e * a.b_idx_s, a.scale_d + e * a.b_scale_d, a.scale_s + e * a.b_scale_s,
                (int)t, (int)(r16 * 16 - t * a.rows), wave, nblk};
      },
      [&](const DecSource& s, int b, DecOperand<F>& o) {
        const bool dense = b < nd;
        const int k = dense ? b : b - nd, nkb = dense ? nd : ns;
        // 32-bit offsets from an expert's buffers
        const uint32_t kb = s.tile * nkb + k, row = kb * a.rows + s.row;
        const uint32_t group = (s.tile * ((nkb + 3) / 4) + k / 4) * a.rows + s.row;
        const uint8_t *val = pick(dense, s.val_d, s.val_s), *scale = pick(dense, s.scale_d, s.scale_s);
        // a dense block has no metadata and reads its values' first bytes
        const uint8_t* meta = pick(dense, s.val_d, s.meta);
        o.index = at<int>(pick(dense, s.idx_d, s.idx_s), dense ? kb * 128 + 4 * (lane & 31) : kb * 256 + 4 * lane);
#pragma unroll
        for (int f = 0; f < F; ++f) {
          o.v[f] = at<fp8_u32x2>(val, row * 32 + 32 * i16 + 8 * kc + 512 * f);
          o.scale[f] = at<uint8_t>(scale, group + 16 * f + i16);
          o.m[f] = at<uint16_t>(meta, row * 8 + 8 * i16 + 2 * kc + 128 * f);
        }
      },
      [&](int b, const DecOperand<F>& o) {
        // the lane's share of the transposed reads: eight tokens of position 8 kc + i16 / 2, and 32 further on (at width
        // 8 the same ones again: columns that nothing reads)
        const int s8 = width == 16 ? 8 * (i16 & 1) : 0, p = 8 * kc + (i16 >> 1);
        const bool dense = b < nd;
        const int row = ((uint32_t)o.index < (uint32_t)a.cin ? o.index : a.cin) * width;
        fp8_u32x2 raw[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int pos = p + 32 * u;
          // a dense block is multiplied as a 2:4 block whose groups keep positions 0 and 1: column 2 q + u at 4 q + u
          raw[u] = tr_read8(slab + __shfl(row, dense ? 2 * (pos >> 2) + (pos & 1) : pos) + s8);
        }
        const bf16x8 lo8 = __builtin_bit_cast(bf16x8, fp8_expand(raw[0], xs)), hi8 = __builtin_bit_cast(bf16x8, fp8_expand(raw[1], xs));
        const bf16x16 bv = __builtin_shufflevector(lo8, hi8, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
        for (int f = 0; f < F; ++f) {
          const bf16x8 av = __builtin_bit_cast(bf16x8, fp8_expand(o.v[f], fp8_scale(o.scale[f])));
          acc[f] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av, bv, acc[f], dense ? 0x4444 : (int)o.m[f], 0, 0);
        }
      },
      [&](int i) {
        const unsigned sg = (mine.first + i) / n_rb;
        rb = mine.first + i - sg * n_rb;
        if ((int)sg != held) {
          held = sg;
          now = next;
          round_x<TOKEN>(a, now, width, v, slab, top, scales);
          step_barrier();
          xs = fp8_scale(scales[i16 & (width - 1)]);
        }
#pragma unroll
        for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
      },
      [&](int) {
        // lane's sums of wave w, fragment f: red[w][f][lane]
        constexpr int kPitch = dec_red_bytes(F) / 4 / kDecWaves, kParts = kDecWaves / F;
#pragma unroll
        for (int f = 0; f < F; ++f) *reinterpret_cast<f32x4*>(red + wave * kPitch + 256 * f + 4 * lane) = acc[f];
        step_barrier();
        const int tid = own_thread();
        const int part = tid % kParts, g = tid / kParts, f = g >> 6, l = g & 63;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < F; ++w) s += *reinterpret_cast<const f32x4*>(red + (part * F + w) * kPitch + 4 * g);
        const int j = l & 15, n0 = now.n0, n1 = now.n1, n = (j < 8 ? n0 : n1 - 8) + j, from = now.lo + (j & 8), row = rb * 16 * F + 16 * f + 4 * (l >> 4);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v = s[q] + quad1(s[q]);
          if (kParts >= 4) v += quad2(v);
          if (kParts == 8) v += octet(v);
          if (q % kParts == part && j < width && n >= from && n < now.hi && n < from + 8) a.y[(int64_t)(row + q) * a.ldy + n] = to_bf16(v);
        }
        step_barrier();
      });
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
  if (ldx >= lim) return fail(HINM_ESHAPE, "ldx=%lld must be below 2^31", (long long)ldx);
  if (n_cols == 0) return HINM_OK;
  if (!x || !y) return fail(HINM_EINVAL, "x and y must be non-NULL");
  if (!hinm::aligned(x, 2) || !hinm::aligned(y, 2)) return fail(HINM_EALIGN, "x and y must be 2-byte aligned");
  return HINM_OK;
}

// Tokens a workgroup of the many-token kernel takes.  256 halves the bytes of
// packed values of 128 but costs an expert with few columns the whole block, and
// one weight of few row blocks half of its workgroups.  Measured, 128 against
// 256: 4096x4096 at 256, 700 and 1500 tokens 29 / 31, 37 / 40, 56 / 49 us; 8
// experts of 11008x4096 with 64, 115, 130 and 500 columns on average 86 / 116,
// 97 / 111, 124 / 108, 275 / 215.
int token_block(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols) {
  const int64_t avg = (n_cols + n_experts - 1) / n_experts;
  if (n_experts == 1) return (p.cout / 64) * ((n_cols + 255) / 256) <= kCus ? 128 : 256;
  return avg <= 112 ? 128 : 256;
}

// Columns of a decode segment, 16, or 8 where 16 do not fit in LDS or one weight
// has no more (of experts, some have more than eight where eight are the
// average: 8 of 11008x4096 51 us, against 41), or 0 where the many-token kernel
// is taken.  Measured, this kernel against the other: one weight of 11008x4096
// at 80 and 128 tokens 29 / 30 and 34 / 31 us, 4096x4096 20 / 26 and 19 / 26,
// 4096x11008 (segments of 8) at 32 and 64 27 / 37 and 44 / 37; 64 experts of
// 1408x2048 with 24 and 32 columns on average 55 / 59 and 66 / 58, 8 of
// 11008x4096 57 / 80 and 72 / 80, 8 of 4096x11008 (segments of 8) with 4, 8 and
// 12 46 / 68, 69 / 68 and 74 / 68.
int decode_width(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols) {
  const int64_t avg = (n_cols + n_experts - 1) / n_experts;
  const int fit = dec_fits(p.cin, 16, 1) ? 16 : dec_fits(p.cin, 8, 1) ? 8 : 0;
  if (fit == 0 || p.cin < 8 || p.n_dense + p.n_24 == 0 || n_cols * (p.cout / 16) >= (int64_t)1 << 31) return 0;
  const int width = n_experts == 1 && n_cols <= 8 ? 8 : fit;
  const int most = n_experts == 1 ? (fit == 16 ? 96 : 32) : (fit == 16 ? 24 : 8);
  return avg <= most ? width : 0;
}

// Workspace: none for few tokens.  Arrival counters and the partial sums of
// kMaxWgs workgroups, where this launch or one of fewer columns may split; then the rounded activations of
// one window of columns (at most 2^30 bytes, a multiple of 256 columns), their
// scales and the pieces' largest magnitudes.
struct Workspace {
  int64_t window, ld8;               // columns of a window, their pitch
  int64_t x8, xs, part, bytes;       // offsets
  int chunks, split;
};
Workspace workspace_of(const hinm_plan_t& p, int32_t n_experts, int64_t n_cols) {
  Workspace w{};
  if (n_cols == 0 || decode_width(p, n_experts, n_cols)) return w;
  w.window = std::min({n_cols, (int64_t)1 << 23, std::max<int64_t>(256, ((int64_t)1 << 30) / p.cin / 256 * 256)});
  w.ld8 = w.window <= 128 ? 128 : ((w.window + 255) / 256 | 1) * 256;
  w.chunks = (int)std::min<int64_t>(kChunks, (p.cin + 63) / 64);
  const int nt = token_block(p, n_experts, n_cols);
  const int64_t fewest = (p.cout / 64) * (n_experts == 1 ? (w.window + nt - 1) / nt : 1);   // items, if any
  w.split = fewest * 2 <= kMaxWgs;
  // Where one weight's smallest launches may split, larger ones keep their room, so that a workspace that serves some
  // columns serves fewer; of experts all may or none.
  const int room = std::max(w.split ? nt : 0, n_experts == 1 && (p.cout / 64) * 2 <= kMaxWgs ? 128 : 0);
  w.x8 = hinm::kWsCounterBytes + (int64_t)kMaxWgs * room * 64 * 4;
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
  const Buf bufs[7] = {
      {k->val_dense, p.bytes_val_dense, "val_dense"}, {k->scale_dense, p.bytes_val_dense, "scale_dense"},
      {k->idx_dense, p.bytes_idx_dense, "idx_dense"}, {k->val_24, p.bytes_val_24, "val_24"},
      {k->scale_24, p.bytes_val_24, "scale_24"}, {k->meta_24, p.bytes_meta_24, "meta_24"}, {k->idx_24, p.bytes_idx_24, "idx_24"}};
  st = check_bufs(bufs, 7, "");
  if (st) return st;
  const Workspace w = workspace_of(p, n_experts, n_cols);
  if (w.bytes > 0 && (!workspace || workspace_bytes < (size_t)w.bytes))
    return fail(HINM_EWORKSPACE, "workspace of %zu bytes given, %lld needed", workspace_bytes, (long long)w.bytes);
  if (w.bytes > 0 && !hinm::aligned(workspace, 256)) return fail(HINM_EALIGN, "workspace is not 256-byte aligned");
  st = hinm::ensure_device();
  if (st) return st;
  char* const ws = static_cast<char*>(workspace);
  auto bytes = [](const void* q) { return static_cast<const uint8_t*>(q); };
  Fp8Args a{};
  a.val_d = k->val_dense;
  a.val_s = k->val_24;
  a.scale_d = k->scale_dense;
  a.scale_s = k->scale_24;
  a.meta = bytes(k->meta_24);
  a.idx_d = bytes(k->idx_dense);
  a.idx_s = bytes(k->idx_24);
  a.nkb_d = p.n_dense_pad / HINM_KB_DENSE;
  a.nkb_s = p.n_24_pad / HINM_KB_24;
  a.b_val_d = p.bytes_val_dense / 2;
  a.b_val_s = p.bytes_val_24 / 2;
  a.b_scale_d = (int64_t)p.cout * ((a.nkb_d + 3) / 4);
  a.b_scale_s = (int64_t)p.cout * ((a.nkb_s + 3) / 4);
  a.b_meta = p.bytes_meta_24;
  a.b_idx_d = p.bytes_idx_dense;
  a.b_idx_s = p.bytes_idx_24;
  a.ldx = ldx;
  a.x8 = bytes(ws + w.x8);
  a.xs = bytes(ws + w.xs);
  a.ld8 = (int)w.ld8;
  a.ldy = ldy;
  a.starts = starts;
  a.counts = counts;
  a.n_experts = n_experts;
  a.total = (int)n_cols;
  a.may_split = w.split;
  a.cin = p.cin;
  a.cout = p.cout;
  a.rows = p.tile_rows;
  a.n_tiles = p.n_tiles;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  if (const int width = decode_width(p, n_experts, n_cols)) {
    a.n_cols = (int)n_cols;
    a.x = static_cast<const uint16_t*>(x);
    a.y = static_cast<uint16_t*>(y);
    // Rows an item, 16 f: those that leave the busiest workgroup the least to do.  An item costs as much as another
    // five fragments of 16 rows (11008x4096 at one token, 3, 2 and 1 items of 1, 2 and 4 fragments: 11.8, 10.7 and
    // 9.3 us; 4096x4096, one item each: 8.0, 8.0 and 8.8).
    const int64_t segs = n_experts == 1 ? (n_cols + width - 1) / width : std::min<int64_t>(n_experts, n_cols);
    auto cost = [&](int f) {
      const int64_t n_rb = p.cout / (16 * f), share = std::max<int64_t>(kCus / segs, 1);
      return dec_fits(p.cin, width, f) ? (n_rb + share - 1) / share * (f + 5) : INT64_MAX;
    };
    const int f = cost(1) <= cost(2) && cost(1) <= cost(4) ? 1 : cost(2) <= cost(4) ? 2 : 4;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(kCus), dim3(kDecThreads), 0, stream, a, width); };
    if (!starts && ldx == 1) f == 4 ? go(fp8_decode_kernel<4, true>) : f == 2 ? go(fp8_decode_kernel<2, true>) : go(fp8_decode_kernel<1, true>);
    else f == 4 ? go(fp8_decode_kernel<4, false>) : f == 2 ? go(fp8_decode_kernel<2, false>) : go(fp8_decode_kernel<1, false>);
    const hipError_t e = hipGetLastError();
    return e == hipSuccess ? HINM_OK : fail(HINM_EHIP, "8-bit product launch: %s", hipGetErrorString(e));
  }
  uint16_t* const tops = reinterpret_cast<uint16_t*>(ws + w.part);
  float* const part = reinterpret_cast<float*>(ws + hinm::kWsCounterBytes);
  unsigned* const counters = reinterpret_cast<unsigned*>(ws);
  const int nt = token_block(p, n_experts, n_cols);
  const hinm::EnqueueLock whole(workspace);
  for (int64_t c0 = 0; c0 < n_cols; c0 += w.window) {
    a.before = (int)c0;
    a.n_cols = (int)std::min(n_cols - c0, w.window);
    a.x = static_cast<const uint16_t*>(x) + c0;
    a.y = static_cast<uint16_t*>(y) + c0;
    const dim3 grid((unsigned)((a.n_cols + 255) / 256), (unsigned)w.chunks);
    hipLaunchKernelGGL(fp8_colmax_kernel, grid, dim3(256), 0, stream, a, tops);
    hipLaunchKernelGGL(fp8_columns_kernel, grid, dim3(256), 0, stream, a, tops, w.chunks,
                       reinterpret_cast<uint8_t*>(ws + w.x8), reinterpret_cast<uint8_t*>(ws + w.xs));
    if (nt == 256) hipLaunchKernelGGL(fp8_prefill_kernel<256>, dim3(kMaxWgs), dim3(kPreThreads), 0, stream, a, part, counters);
    else hipLaunchKernelGGL(fp8_prefill_kernel<128>, dim3(kMaxWgs), dim3(kPreThreads), 0, stream, a, part, counters);
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
