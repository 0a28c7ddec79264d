// hinm_moe_layer: a gated mixture-of-experts layer for a few tokens in two
// kernels (formulas at hinm_moe_layer).
//
// A few tokens make a layer a read of the chosen experts' packed weights, so
// both kernels are built around that stream.  The activations of a segment -
// up to 16 of an expert's tokens - are held in LDS whole, [channel][token], so
// that the channels a tile keeps are gathered there: the transposed LDS read
// takes an address a lane, which is the channel's row.  The gather therefore
// costs no memory access and no staging, every global load of a wave (index
// words, values, metadata) is at an address known beforehand, and 16 waves a
// compute unit each keep their own K-blocks in flight.
//
//   up kernel    every workgroup works out the routing from the logits, then
//                takes (segment, 64 rows of the inner channels): eight waves
//                the gate's K-blocks, eight the up projection's; the sums meet
//                in LDS and become h, which goes to the workspace laid out as
//                the down kernel's LDS rows.
//   down kernel  a workgroup takes 64 rows of Y and a share of all segments'
//                K-blocks; each segment's sums are multiplied by the router's
//                weights and added to the tokens' in LDS, and the shares meet
//                in the workspace.
//
// h is a matrix operand and so bf16, but rounded once it would cost the output
// as much as its own rounding (relative error of the layer 0.0024, against
// 0.0017 from the rounding of Y alone).  It is held as the sum of two bf16
// values instead, its rounding and what that leaves, in two columns of the
// matrix instruction, of which a few tokens leave many idle.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "hinm_device.h"
#include "hinm_fp8.h"
#include "hinm_internal.h"
#include "hinm_mx4.h"
#include "hinm_ragged.h"

using hinm::fail;

namespace {

constexpr int kWaves = 16;                         // of a workgroup; one workgroup a compute unit
constexpr int kThreads = 64 * kWaves;
constexpr int kTokens = HINM_MOE_MAX_TOKENS;
constexpr int kPairs = kTokens * HINM_MAX_TOP_K;   // (token, expert) pairs at most; a segment holds at least one
constexpr int kSlab = 131328;                      // bytes of LDS for a segment's activations and a row of zeros
constexpr int kMaxChannels = 16384;                // of four columns, with the row of zeros
static_assert((kMaxChannels + 1) * 8 <= kSlab, "four columns of the most channels fit");
constexpr int kRed = 260;                          // floats between the waves' sums: 256, and conflict-free reads

// One stack of packed weights; strides are bytes of one expert.
struct MoeStack {
  const uint8_t *val_d, *val_s, *scale_d, *scale_s, *meta, *idx_d, *idx_s;
  int64_t b_val_d, b_val_s, b_scale_d, b_scale_s, b_meta, b_idx_d, b_idx_s;
  int rows, nkb_d, nkb_s, cin, cout;
};

// A segment: n of an expert's tokens from the rank0-th on.
struct Seg {
  uint16_t expert, slot;           // slot: of its first token
  uint8_t n, rank0, count, pad;    // count: tokens of the expert
  uint16_t down;                   // the expert's first segment of the down kernel
};

// What the up kernel leaves for the down kernel: its segments as expert, first
// slot (10 bits each) and tokens, and the tokens and weights by slot.
struct Table {
  int n_seg;
  uint32_t seg[kPairs];
  uint16_t token[kPairs];
  float weight[kPairs];
};

struct MoeArgs {
  const void* logits;
  const uint16_t* x;
  uint16_t* y;
  Table* table;
  uint16_t* h;                     // [segment][inner channels][tokens]
  float* part;
  unsigned* counters;
  int64_t ldl, ldx, ldy, h_seg;    // h_seg: elements between segments
  int logits_fp32, n_tokens, n_experts, top_k, renormalize, up_cap, down_cap;
  MoeStack gate, up, down;
};

// Columns a row of the slab holds for n of them: 8 bytes are the least a
// transposed read takes.
__device__ inline int row_columns(int n) { return n <= 4 ? 4 : n <= 8 ? 8 : 16; }

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// One K-block's operands of a lane: the fragments (16 rows each) of an item.
template <int VALUES, int F>
struct Operand {                   // bf16
  u32x4 v[F];
  uint32_t m[F];
  int index;
};
template <int F>
struct Operand<HINM_VALUES_MX4, F> {
  uint32_t v[F];
  uint32_t scale, m[F / 2];        // scale: a byte a fragment; m: 16 bits a fragment
  int index;
};
template <int F>
struct Operand<HINM_VALUES_FP8, F> {
  u32x2 v[F];
  uint32_t m[F], scale[F];
  int index;
};

// An item: 16 F rows of one expert's weight over K-blocks b0 .. b1 - 1.
struct Item {
  int expert, rows16, b0, b1;      // rows16: its first row / 16
};

// Where a wave reads an item's operands; all scalars.
struct Source {
  const uint8_t *val_d, *val_s, *meta, *idx_d, *idx_s, *scale_d, *scale_s;
  int tile, row;                   // tile, and the item's first row in it
  int first, end;                  // the wave's blocks: first, first + nw, ... below end
};

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ inline Source source_of(const MoeStack& w, const Item& it, int v) {
  const int t = it.rows16 * 16 / w.rows;
  const int64_t e = it.expert;
  return {w.val_d + e * w.b_val_d, w.val_s + e * w.b_val_s, w.meta + e * w.b_meta, w.idx_d + e * w.b_idx_d,
          w.idx_s + e * w.b_idx_s, w.scale_d + e * w.b_scale_d, w.scale_s + e * w.b_scale_s,
          t, it.rows16 * 16 - t * w.rows, it.b0 + v, it.b1};
}

template <class T>
__device__ inline T at(const uint8_t* base, uint32_t offset) { return *reinterpret_cast<const T*>(base + offset); }

// Block b's operands.  The block's place is scalar and the lane's share a
// constant; a dense block has no metadata and reads its values' bytes instead.
template <int VALUES, int F>
__device__ inline void load_block(const MoeStack& w, const Source& s, int b, Operand<VALUES, F>& o) {
  const uint32_t lane = threadIdx.x & 63, i16 = lane & 15, kc = lane >> 4;
  const bool dense = b < w.nkb_d;
  const int k = dense ? b : b - w.nkb_d;
  const int64_t kb = (int64_t)s.tile * (dense ? w.nkb_d : w.nkb_s) + k;
  o.index = dense ? at<int>(s.idx_d + kb * 128, 4 * (lane & 31)) : at<int>(s.idx_s + kb * 256, 4 * lane);
  if constexpr (VALUES == HINM_VALUES_MX4) {
    const int64_t u = kb * (w.rows / 64) + s.row / 64;
    const uint8_t* val = (dense ? s.val_d : s.val_s) + u * 1024;
    const uint32_t f0 = (uint32_t)(s.row >> 4) & 3;          // 0 or 2 with two fragments
    o.scale = at<uint32_t>((dense ? s.scale_d : s.scale_s) + u * 64, 4 * i16) >> (8 * f0);
    const uint8_t* meta = dense ? val : s.meta + u * 512;
    if constexpr (F == 4) {
      const u32x4 v = at<u32x4>(val, 256 * kc + 16 * i16);
      const u32x2 m = at<u32x2>(meta, 128 * kc + 8 * i16);
      for (int f = 0; f < 4; ++f) o.v[f] = v[f];
      o.m[0] = m[0];
      o.m[1] = m[1];
    } else {
      const u32x2 v = at<u32x2>(val, 256 * kc + 16 * i16 + 4 * f0);
      o.v[0] = v[0];
      o.v[1] = v[1];
      o.m[0] = at<uint32_t>(meta, 128 * kc + 8 * i16 + 2 * f0);
    }
  } else {
    constexpr int kRow = VALUES == HINM_VALUES_FP8 ? 32 : 64;      // bytes of a row
    const int64_t row = kb * w.rows + s.row;
    const uint8_t* val = (dense ? s.val_d : s.val_s) + row * kRow;
    const uint8_t* meta = dense ? val : s.meta + row * 8;
    const int64_t group = (int64_t)s.tile * (((dense ? w.nkb_d : w.nkb_s) + 3) / 4) + k / 4;
    const uint8_t* scale = (dense ? s.scale_d : s.scale_s) + group * w.rows + s.row;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (VALUES == HINM_VALUES_FP8) {
        o.v[f] = at<u32x2>(val, 32 * i16 + 8 * kc + 512 * f);
        o.scale[f] = at<uint8_t>(scale, 16 * f + i16);
      } else {
        o.v[f] = at<u32x4>(val, 64 * i16 + 16 * kc + 1024 * f);
      }
      o.m[f] = at<uint16_t>(meta, 8 * i16 + 2 * kc + 128 * f);
    }
  }
}

// acc += the block's rows x 16 columns of the slab: rows of `pitch` bytes,
// zeros in row cin.
template <int VALUES, int F>
__device__ inline void multiply_block(const MoeStack& w, int b, const Operand<VALUES, F>& o, const uint8_t* slab,
                                      int pitch, f32x4 (&acc)[F]) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, kc = lane >> 4;
  // The lane's share of the transposed reads: 8 bytes of columns 4 s .. 4 s + 3
  // (past a short row the first ones again: columns that nothing reads) of
  // positions 8 kc + i16 / 4 + {0, 4, 32, 36}.
  const int s8 = 8 * min(i16 & 3, pitch / 8 - 1), p0 = 8 * kc + (i16 >> 2);
  const bool dense = b < w.nkb_d;
  const int row = (o.index < 0 || o.index >= w.cin ? w.cin : o.index) * pitch;
  v4i16 q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int p = p0 + 4 * (k & 1) + 32 * (k >> 1);
    // a dense block is multiplied as a 2:4 block whose groups keep positions 0 and 1: column 2 q + u at 4 q + u
    q[k] = tr_read_b(slab + __shfl(row, dense ? 2 * (p >> 2) + (p & 1) : p) + s8);
  }
  const bf16x8 lo8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(q[0], q[1], 0, 1, 2, 3, 4, 5, 6, 7));
  const bf16x8 hi8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(q[2], q[3], 0, 1, 2, 3, 4, 5, 6, 7));
  const bf16x16 bv = __builtin_shufflevector(lo8, hi8, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
  for (int f = 0; f < F; ++f) {
    bf16x8 av;
    int sidx;
    if constexpr (VALUES == HINM_VALUES_MX4) {
      av = mx4_expand(o.v[f], mx4_scale((o.scale >> (8 * f)) & 255u));
      sidx = (int)((o.m[f >> 1] >> (16 * (f & 1))) & 0xffffu);
    } else if constexpr (VALUES == HINM_VALUES_FP8) {
      av = __builtin_bit_cast(bf16x8, fp8_expand(o.v[f], fp8_scale(o.scale[f])));
      sidx = (int)o.m[f];
    } else {
      av = __builtin_bit_cast(bf16x8, o.v[f]);
      sidx = (int)o.m[f];
    }
    acc[f] = __builtin_amdgcn_smfmac_f32_16x16x64_bf16(av, bv, acc[f], dense ? 0x4444 : sidx, 0, 0);
  }
}

// The wave's share - blocks v, v + NW, ... - of `items` items, in one stream:
// while a pair of blocks is multiplied the next pair's operands are on their
// way, across the items' ends too.  item_of(i) names an item (with one block at
// least) without reading memory, begin(i) makes
// its activations ready (in step for the whole workgroup) and returns their
// pitch, and finish(i, acc) takes its sums (in step, too).  One loop body for
// the first loads, the products and the items' ends: a launch reads every
// instruction from memory once, and these kernels last some ten times that.
template <int VALUES, int F, int NW, class ItemOf, class Begin, class Finish>
__device__ inline void stream(const MoeStack& w, int items, int v, const uint8_t* slab, ItemOf item_of, Begin begin,
                              Finish finish) {
  if (items <= 0) return;
  Operand<VALUES, F> o[2];
  int block[2] = {-1, -1};         // the operands' blocks; -1: none
  Source src{};
  int ahead = -1, pairs = 0;       // the item that loads are at, and its pairs left
  int pitch = 8;
  f32x4 acc[F];
#pragma unroll
  for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma nounroll
  while (true) {
    const bool enter = pairs == 0;
    if (enter) {
      pairs = 1;
      if (++ahead < items) {
        src = source_of(w, item_of(ahead), v);
        pairs = max(1, (src.end - src.first + 2 * NW - 1) / (2 * NW));
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (block[k] >= 0) multiply_block<VALUES, F>(w, block[k], o[k], slab, pitch, acc);
      // past its end an item's last block is read again: a load that only sometimes happens would make every wait one
      // for all loads in flight
      const int b = min(src.first, src.end - 1);
      load_block<VALUES, F>(w, src, b, o[k]);
      block[k] = src.first < src.end ? b : -1;
      src.first += NW;
    }
    --pairs;
    if (enter) {
      if (ahead > 0) finish(ahead - 1, acc);
      if (ahead >= items) return;
      pitch = begin(ahead);
#pragma unroll
      for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
}

// The waves' sums of the rows r0 .. r0 + 256 / width - 1 (of 16 F) in `width`
// columns: put by each wave, summed over four waves by each thread, which has
// element threadIdx.x / 4 and waves 4 (threadIdx.x % 4) .. + 3.
template <int F>
__device__ inline void put_sums(float* red, const f32x4 (&acc)[F], int r0, int width) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15;
#pragma unroll
  for (int f = 0; f < F; ++f)
    if (16 * f >= r0 && 16 * f < r0 + 256 / width && col < width)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[wave * kRed + (16 * f - r0 + 4 * (lane >> 4) + q) * width + col] = acc[f][q];
}
__device__ inline float four_sums(const float* red) {
  const float* p = red + (threadIdx.x & 3) * 4 * kRed + (threadIdx.x >> 2);
  return (p[0] + p[kRed]) + (p[2 * kRed] + p[3 * kRed]);
}
// The value of lane ^ 1 or ^ 2.
__device__ inline float quad1(float v) { return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xf, 0xf, true)); }
__device__ inline float quad2(float v) { return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xf, 0xf, true)); }

// A segment's scalars.
__device__ inline Seg uniform_seg(const Seg& s) {
  return {(uint16_t)uniform(s.expert), (uint16_t)uniform(s.slot), (uint8_t)uniform(s.n), (uint8_t)uniform(s.rank0),
          (uint8_t)uniform(s.count), 0, (uint16_t)uniform(s.down)};
}

// ---------------------------------------------------------------------------
// Routing of all tokens, by every workgroup for itself: a wave takes a token.
// ---------------------------------------------------------------------------
struct RouteScratch {
  uint32_t mask[HINM_MAX_EXPERTS];       // tokens of every expert
  uint16_t start[HINM_MAX_EXPERTS];      // its first slot
  int16_t id[kPairs];
  float weight[kPairs];
};

// A logit as a whole number of the same order, 0 for what is not eligible; and
// back.
__device__ inline uint32_t key_of(float l) {
  l += 0.f;                                        // -0 is 0
  const uint32_t u = __float_as_uint(l);
  return l > -__builtin_inff() ? ((int)u < 0 ? ~u : u | 0x80000000u) : 0u;
}
__device__ inline float logit_of(uint32_t key) { return __uint_as_float((int)key < 0 ? key & 0x7fffffffu : ~key); }

// The wave's largest key (lane 63 of a chain of shifts within rows of 16 and
// broadcasts between them), and the wave's sum.
template <int CTRL>
__device__ inline uint32_t shifted(uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false); }
__device__ inline uint32_t wave_max(uint32_t v) {
  v = max(v, shifted<0x111>(v));
  v = max(v, shifted<0x112>(v));
  v = max(v, shifted<0x114>(v));
  v = max(v, shifted<0x118>(v));
  v = max(v, shifted<0x142>(v));
  v = max(v, shifted<0x143>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ inline float wave_sum(float v) {
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
  return v;
}

// Token n's experts and weights; NL keys a lane, expert 64 i + lane.
template <int NL>
__device__ inline void route_token(const MoeArgs& a, RouteScratch& r, int n) {
  const int lane = threadIdx.x & 63;
  uint32_t raw[NL];
  if (a.logits_fp32) {
#pragma unroll
    for (int i = 0; i < NL; ++i) raw[i] = static_cast<const uint32_t*>(a.logits)[min(64 * i + lane, a.n_experts - 1) * a.ldl + n];
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) raw[i] = static_cast<const uint16_t*>(a.logits)[min(64 * i + lane, a.n_experts - 1) * a.ldl + n];
  }
  uint32_t key[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) key[i] = 64 * i + lane < a.n_experts ? key_of(__uint_as_float(a.logits_fp32 ? raw[i] : raw[i] << 16)) : 0u;
  float top = 0.f, sum = 0.f, mine = 0.f;          // mine: lane j's exp(l_j - top)
  int chosen = -1;                                 // lane j's expert
#pragma nounroll
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = key[0];
#pragma unroll
    for (int i = 1; i < NL; ++i) best = max(best, key[i]);
    best = wave_max(best);
    if (best == 0u) break;
    int id = -1;
#pragma unroll
    for (int i = NL - 1; i >= 0; --i) {
      const uint64_t who = __ballot(key[i] == best);
      if (who) id = 64 * i + __builtin_ctzll(who);
    }
    const float l = logit_of(best);
    if (j == 0) {
      top = l;
      if (!a.renormalize) {
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const float li = logit_of(key[i]);
          sum += key[i] == 0u ? 0.f : li == top ? 1.f : expf(li - top);
        }
        sum = wave_sum(sum);
      }
    }
    const float p = l == top ? 1.f : expf(l - top);
    if (a.renormalize) sum += p;
    if (lane == j) mine = p, chosen = id;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (64 * i + lane == id) key[i] = 0u;
  }
  if (lane < a.top_k) {
    r.id[n * a.top_k + lane] = (int16_t)chosen;
    r.weight[n * a.top_k + lane] = chosen >= 0 ? mine / sum : 0.f;
    if (chosen >= 0) atomicOr(&r.mask[chosen], 1u << n);
  }
}

// The up kernel's segments and their tokens by slot go to `seg` and `token`,
// their number to n_seg; down (one workgroup's): the table for the down kernel.
__device__ inline void route_tokens(const MoeArgs& a, RouteScratch& r, int* n_seg, Seg* seg, uint16_t* token, Table* down) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  for (int e = threadIdx.x; e < a.n_experts; e += kThreads) r.mask[e] = 0u;
  __syncthreads();
  for (int n = wave; n < a.n_tokens; n += kWaves) {
    if (a.n_experts <= 64) route_token<1>(a, r, n);
    else if (a.n_experts <= 256) route_token<4>(a, r, n);
    else route_token<HINM_MAX_EXPERTS / 64>(a, r, n);
  }
  __syncthreads();
  // slots by expert and token, and the segments of both kernels; the three running counts (each at most kPairs) share
  // a word
  if (wave == 0) {
    uint32_t before = 0;                           // counts of the experts before
#pragma nounroll
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < a.n_experts ? __popc(r.mask[e]) : 0;
      const int nu = (c + a.up_cap - 1) / a.up_cap, nd = (c + a.down_cap - 1) / a.down_cap;
      const uint32_t own = (uint32_t)c | (uint32_t)nu << 10 | (uint32_t)nd << 20;
      uint32_t all = own;
      for (int d = 1; d < 64; d *= 2) {
        const uint32_t v = __shfl_up(all, d);
        if (lane >= d) all += v;
      }
      const uint32_t at = before + all - own;
      const int s0 = at & 1023, u0 = at >> 10 & 1023, d0 = at >> 20;
      if (e < a.n_experts) r.start[e] = (uint16_t)s0;
      for (int q = 0; q < nu; ++q)
        seg[u0 + q] = {(uint16_t)e, (uint16_t)(s0 + q * a.up_cap), (uint8_t)min(a.up_cap, c - q * a.up_cap),
                       (uint8_t)(q * a.up_cap), (uint8_t)c, 0, (uint16_t)d0};
      if (down)
        for (int q = 0; q < nd; ++q)
          down->seg[d0 + q] = (uint32_t)e | (uint32_t)(s0 + q * a.down_cap) << 10 | (uint32_t)min(a.down_cap, c - q * a.down_cap) << 20;
      before += __shfl(all, 63);
    }
    if (lane == 0) {
      *n_seg = before >> 10 & 1023;
      if (down) down->n_seg = before >> 20;
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < a.n_tokens * a.top_k) {
    const int e = r.id[threadIdx.x], n = threadIdx.x / a.top_k;
    if (e >= 0) {
      const int slot = r.start[e] + __popc(r.mask[e] & ((1u << n) - 1u));
      token[slot] = (uint16_t)n;
      if (down) {
        down->token[slot] = (uint16_t)n;
        down->weight[slot] = r.weight[threadIdx.x];
      }
    }
  }
  __syncthreads();
}

// A segment's tokens from X into the slab, [channel][column], and the row of
// zeros.  A thread reads eight tokens of a channel at once and writes those of
// the segment, four channels in flight.
__device__ inline void load_tokens(const MoeArgs& a, const Seg& seg, const uint16_t* token, uint16_t* slab) {
  const int cin = a.up.cin, width = row_columns(seg.n);
  uint32_t mask = 0;
  for (int j = 0; j < seg.n; ++j) mask |= 1u << token[seg.slot + j];
  mask = (uint32_t)uniform((int)mask);
  const int64_t end = (int64_t)(cin - 1) * a.ldx + a.n_tokens;       // elements of X
  constexpr int U = 4;
  int col = 0;
  for (int g = 0; g < 32; g += 8) {
    const uint32_t some = (mask >> g) & 255u;
    if (!some) continue;
    for (int c0 = threadIdx.x; c0 < cin; c0 += U * kThreads) {
      u32x4 v[U];
      int past[U];                 // elements that the load begins before its own, at the end of X
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = (int64_t)min(c0 + u * kThreads, cin - 1) * a.ldx + g;
        const int64_t from = min(at, end - 8);     // X has 64 elements or more
        past[u] = (int)(at - from);
        v[u] = *reinterpret_cast<const any_u32x4*>(a.x + from);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (past[u] & 4) v[u][0] = v[u][2], v[u][1] = v[u][3];
        if (past[u] & 2) v[u][0] = v[u][1], v[u][1] = v[u][2], v[u][2] = v[u][3];
        if (past[u] & 1)
#pragma unroll
          for (int k = 0; k < 4; ++k) v[u][k] = v[u][k] >> 16 | (k < 3 ? v[u][k + 1] << 16 : 0u);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * kThreads;
        if (c >= cin) continue;
        int j = col;
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if ((some >> t) & 1u) slab[c * width + j++] = (uint16_t)(v[u][t >> 1] >> (16 * (t & 1)));
      }
    }
    col += __popc(some);
  }
  if ((int)threadIdx.x < width) slab[cin * width + threadIdx.x] = 0;
}

// Items are (segment, 32 rows of the inner channels), a contiguous range of
// them a workgroup: of 64 rows, the 344 items of a token's two experts of 11008
// channels left the busiest of 256 workgroups two.
template <int VALUES>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
  constexpr int F = 2, R = 16 * F;
  __shared__ __attribute__((aligned(16))) uint8_t slab[kSlab];
  __shared__ __attribute__((aligned(16))) union {
    float red[kWaves * kRed];
    RouteScratch route;
  } sh;
  __shared__ int n_seg;
  __shared__ Seg segs[kPairs];
  __shared__ uint16_t token[kPairs];
  route_tokens(a, sh.route, &n_seg, segs, token, blockIdx.x == 0 ? a.table : nullptr);

  const int wave = uniform(threadIdx.x >> 6);
  const int n_rb = a.up.cout / R, all = uniform(n_seg) * n_rb;     // at most 512 * 512
  const int i0 = (int)((int64_t)blockIdx.x * all / kCus), i1 = (int)((int64_t)(blockIdx.x + 1) * all / kCus);
  const MoeStack& w = wave < kWaves / 2 ? a.gate : a.up;
  int held = -1;
  Seg seg{};                       // of the item at hand
  int rb = 0;
  stream<VALUES, F, kWaves / 2>(
      w, i1 - i0, wave % (kWaves / 2), slab,
      [&](int i) -> Item {
        const int sg = (i0 + i) / n_rb;
        return {uniform(segs[sg].expert), (i0 + i - sg * n_rb) * F, 0, w.nkb_d + w.nkb_s};
      },
      [&](int i) {
        const int sg = (i0 + i) / n_rb;
        rb = i0 + i - sg * n_rb;
        if (sg != held) {
          seg = uniform_seg(segs[sg]);
          __syncthreads();
          load_tokens(a, seg, token, reinterpret_cast<uint16_t*>(slab));
          __syncthreads();
          held = sg;
        }
        return 2 * row_columns(seg.n);
      },
      [&](int, f32x4 (&acc)[F]) {
        const int width = row_columns(seg.n);
#pragma nounroll
        for (int r0 = 0; r0 < R; r0 += 256 / width) {
          put_sums<F>(sh.red, acc, r0, width);
          __syncthreads();
          // of four adjacent threads the first two have the gate's sum, the others the up projection's
          float g = four_sums(sh.red);
          g += quad1(g);
          const float u = quad2(g);
          const int e = threadIdx.x >> 2, row = r0 + e / width, col = e % width;
          if ((threadIdx.x & 3) == 0 && col < seg.n && row < R) {
            // where the down kernel's segment of this token has it
            const int rank = seg.rank0 + col, q = rank / a.down_cap;
            const int wide = row_columns(2 * min(a.down_cap, seg.count - q * a.down_cap));
            const float h = g / (1.f + expf(-g)) * u;
            const uint16_t hi = to_bf16(h);
            uint16_t* dst = a.h + (seg.down + q) * a.h_seg + (int64_t)(rb * R + row) * wide + rank - q * a.down_cap;
            dst[0] = hi;
            dst[wide / 2] = to_bf16(h - __uint_as_float((uint32_t)hi << 16));
          }
          __syncthreads();
        }
      });
}

template <int VALUES>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
  constexpr int F = 4;
  __shared__ __attribute__((aligned(16))) uint8_t slab[kSlab];
  __shared__ float red[kWaves * kRed];
  __shared__ float out[64 * kTokens];
  __shared__ Table table;
  __shared__ int s_last;
  static_assert(sizeof(Table) % 4 == 0 && sizeof(Table) / 4 <= 2 * kThreads, "the table is two words a thread");
#pragma unroll
  for (int q = threadIdx.x; q < (int)sizeof(Table) / 4; q += kThreads)
    reinterpret_cast<uint32_t*>(&table)[q] = reinterpret_cast<const uint32_t*>(a.table)[q];
  __syncthreads();
  const int wave = uniform(threadIdx.x >> 6);
  const int n_rb = a.down.cout / 64, nblk = a.down.nkb_d + a.down.nkb_s, n_seg = uniform(table.n_seg);
  const int units = n_seg * nblk;
  // shares of a row block's K-blocks: as many as leave no compute unit idle, and a block for each wave
  const int splits = max(1, min(kCus / n_rb, units / kWaves));
#pragma nounroll
  for (int item = blockIdx.x; item < n_rb * splits; item += kCus) {
    const int rb = item / splits, split = item % splits;
    // whole segments in turn (an expert's are adjacent: they share its weights in the caches), then an even share of
    // the remaining ones' blocks
    const int rounds = n_seg / splits, rest = (n_seg - rounds * splits) * nblk, r0 = rounds * splits * nblk;
    const int u0 = r0 + split * rest / splits, u1 = r0 + (split + 1) * rest / splits;
    const int s0 = u0 / nblk, parts = u0 < u1 ? (u1 - 1) / nblk - s0 + 1 : 0;
    for (int q = threadIdx.x; q < 64 * kTokens; q += kThreads) out[q] = 0.f;
    auto seg_of = [&](int i) { return i < rounds ? i * splits + split : s0 + i - rounds; };
    int n = 0, slot = 0;           // tokens of the segment at hand, and the first one's slot
    stream<VALUES, F, kWaves>(
        a.down, rounds + parts, wave, slab,
        [&](int i) -> Item {
          const int sg = seg_of(i);
          return {uniform(table.seg[sg] & 1023), rb * F, i < rounds ? 0 : max(0, u0 - sg * nblk),
                  i < rounds ? nblk : min(nblk, u1 - sg * nblk)};
        },
        [&](int i) {
          const int sg = seg_of(i), word = uniform((int)table.seg[sg]);
          slot = word >> 10 & 1023;
          n = word >> 20;
          const int pitch = 2 * row_columns(2 * n);
          const u32x4* src = reinterpret_cast<const u32x4*>(a.h + sg * a.h_seg);
          const int words = a.down.cin * pitch / 16;         // cin is a multiple of 64
          __syncthreads();
          constexpr int U = 4;
#pragma nounroll
          for (int q0 = threadIdx.x; q0 < words; q0 += U * kThreads) {
            u32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = src[min(q0 + u * kThreads, words - 1)];
#pragma unroll
            for (int u = 0; u < U; ++u)
              if (q0 + u * kThreads < words) reinterpret_cast<u32x4*>(slab)[q0 + u * kThreads] = v[u];
          }
          if ((int)threadIdx.x < pitch / 2) reinterpret_cast<uint16_t*>(slab)[a.down.cin * (pitch / 2) + threadIdx.x] = 0;
          __syncthreads();
          return pitch;
        },
        [&](int, f32x4 (&acc)[F]) {
          const int width = row_columns(2 * n);
#pragma nounroll
          for (int r = 0; r < 64; r += 256 / width) {
            put_sums<F>(red, acc, r, width);
            __syncthreads();
            float s = four_sums(red);
            s += quad1(s);
            s += quad2(s);
            s += __shfl_xor(s, 2 * width);                   // the other of the token's two columns
            const int e = threadIdx.x >> 2, row = r + e / width, col = e % width;
            if ((threadIdx.x & 3) == 0 && col < n) out[row * kTokens + table.token[slot + col]] += table.weight[slot + col] * s;
            __syncthreads();
          }
        });
    __syncthreads();
    constexpr int N = 64 * kTokens / kThreads;     // outputs a thread
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = out[k * kThreads + threadIdx.x];
    bool last = true;
    if (splits > 1) {
      float* my = a.part + (int64_t)item * 64 * kTokens + threadIdx.x;
#pragma unroll
      for (int k = 0; k < N; ++k) __hip_atomic_store(my + k * kThreads, v[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (threadIdx.x == 0) s_last = arrive(a.counters + rb, splits);
      __syncthreads();
      last = s_last;
      if (last) {
        const float* p0 = a.part + (int64_t)rb * splits * 64 * kTokens + threadIdx.x;
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = 0.f;
#pragma unroll 4
        for (int s = 0; s < splits; ++s)
#pragma unroll
          for (int k = 0; k < N; ++k)
            v[k] += __hip_atomic_load(p0 + (int64_t)s * 64 * kTokens + k * kThreads, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (last)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int q = k * kThreads + threadIdx.x, row = q / kTokens, col = q % kTokens;
        if (col < a.n_tokens) a.y[((int64_t)rb * 64 + row) * a.ldy + col] = to_bf16(v[k]);
      }
    __syncthreads();
  }
}

// Columns a segment holds at most: as many as fit in LDS.  A token takes one in
// the up kernel and two in the down kernel.
int columns_of(int channels) { return (channels + 1) * 32 <= kSlab ? 16 : (channels + 1) * 16 <= kSlab ? 8 : 4; }

struct Workspace {
  int64_t table, part, h, h_seg, bytes;            // offsets; h_seg in elements
};
Workspace workspace_of(int hidden, int inter, int32_t n_experts, int64_t n_tokens, int32_t top_k) {
  Workspace w{};
  if (n_tokens == 0) return w;
  const int64_t pairs = n_tokens * top_k, columns = columns_of(inter);
  const int64_t segs = std::min(pairs, std::min<int64_t>(n_experts, pairs) + pairs / (columns / 2));
  w.table = hinm::kWsCounterBytes;
  w.part = w.table + (int64_t)((sizeof(Table) + 255) / 256 * 256);
  const int64_t items = std::max<int64_t>(kCus, hidden / 64);
  w.h = w.part + items * 64 * kTokens * 4;
  w.h_seg = (int64_t)inter * columns;
  w.bytes = w.h + (segs * w.h_seg * 2 + 255) / 256 * 256;
  return w;
}

int check_shapes(const hinm_plan_t& up, const hinm_plan_t& down, int32_t n_experts, int64_t n_tokens, int32_t top_k) {
  if (up.tile_rows % 64 != 0 || down.tile_rows % 64 != 0)
    return fail(HINM_ESHAPE, "tile_rows=%d and %d must be multiples of 64", up.tile_rows, down.tile_rows);
  if (down.cout != up.cin || down.cin != up.cout)
    return fail(HINM_ESHAPE, "down is [%d x %d]; [%d x %d] is needed", down.cout, down.cin, up.cin, up.cout);
  if (up.n_dense + up.n_24 == 0 || down.n_dense + down.n_24 == 0) return fail(HINM_ESHAPE, "a projection keeps no value");
  if (up.cin > kMaxChannels || up.cout > kMaxChannels)
    return fail(HINM_ESHAPE, "%d hidden and %d inner channels; at most %d are supported", up.cin, up.cout, kMaxChannels);
  if (n_experts < 1 || n_experts > HINM_MAX_EXPERTS)
    return fail(HINM_ESHAPE, "n_experts=%d; 1 to %d are supported", n_experts, HINM_MAX_EXPERTS);
  if (top_k < 1 || top_k > HINM_MAX_TOP_K || top_k > n_experts)
    return fail(HINM_ESHAPE, "top_k=%d; 1 to %d of the %d experts", top_k, HINM_MAX_TOP_K, n_experts);
  if (n_tokens < 0 || n_tokens > kTokens) return fail(HINM_ESHAPE, "%lld tokens; 0 to %d are supported", (long long)n_tokens, kTokens);
  const int64_t lim = (int64_t)1 << 31;
  for (const hinm_plan_t* p : {&up, &down})
    if (p->bytes_val_dense >= lim || p->bytes_val_24 >= lim)
      return fail(HINM_ESHAPE, "each expert's buffers must be below 2^31 bytes");
  return HINM_OK;
}

struct Buf {
  const void* ptr;
  int64_t bytes;
  const char* name;
};

// Checks one stack and fills in its kernel view.
int stack_of(const char* whose, const hinm_plan_t& p, int32_t values, const void* stack, MoeStack& s) {
  s = MoeStack{};
  s.rows = p.tile_rows;
  s.nkb_d = p.n_dense_pad / HINM_KB_DENSE;
  s.nkb_s = p.n_24_pad / HINM_KB_24;
  s.cin = p.cin;
  s.cout = p.cout;
  s.b_val_d = p.bytes_val_dense;
  s.b_val_s = p.bytes_val_24;
  s.b_meta = p.bytes_meta_24;
  s.b_idx_d = p.bytes_idx_dense;
  s.b_idx_s = p.bytes_idx_24;
  auto fill = [&](const void* vd, const void* sd, const void* id, const void* vs, const void* ss, const void* m,
                  const void* is) {
    s.val_d = static_cast<const uint8_t*>(vd);
    s.val_s = static_cast<const uint8_t*>(vs);
    s.scale_d = static_cast<const uint8_t*>(sd);
    s.scale_s = static_cast<const uint8_t*>(ss);
    s.meta = static_cast<const uint8_t*>(m);
    s.idx_d = static_cast<const uint8_t*>(id);
    s.idx_s = static_cast<const uint8_t*>(is);
  };
  if (values == HINM_VALUES_BF16) {
    const hinm_packed_t* k = static_cast<const hinm_packed_t*>(stack);
    fill(k->val_dense, nullptr, k->idx_dense, k->val_24, nullptr, k->meta_24, k->idx_24);
  } else if (values == HINM_VALUES_MX4) {
    const hinm_mx4_t* k = static_cast<const hinm_mx4_t*>(stack);
    fill(k->val_dense, k->scale_dense, k->idx_dense, k->val_24, k->scale_24, k->meta_24, k->idx_24);
    s.b_val_d /= 4;
    s.b_val_s /= 4;
    s.b_scale_d = s.b_val_d / 16;
    s.b_scale_s = s.b_val_s / 16;
  } else {
    const hinm_fp8_t* k = static_cast<const hinm_fp8_t*>(stack);
    fill(k->val_dense, k->scale_dense, k->idx_dense, k->val_24, k->scale_24, k->meta_24, k->idx_24);
    s.b_val_d /= 2;
    s.b_val_s /= 2;
    s.b_scale_d = (int64_t)p.cout * ((s.nkb_d + 3) / 4);
    s.b_scale_s = (int64_t)p.cout * ((s.nkb_s + 3) / 4);
  }
  const Buf b[7] = {{s.val_d, s.b_val_d, "val_dense"}, {s.scale_d, s.b_scale_d, "scale_dense"}, {s.idx_d, s.b_idx_d, "idx_dense"},
                    {s.val_s, s.b_val_s, "val_24"}, {s.scale_s, s.b_scale_s, "scale_24"}, {s.meta, s.b_meta, "meta_24"},
                    {s.idx_s, s.b_idx_s, "idx_24"}};
  for (const Buf& q : b) {
    if (q.bytes > 0 && !q.ptr) return fail(HINM_EINVAL, "%s: %s is NULL but holds %lld bytes", whose, q.name, (long long)q.bytes);
    if (!hinm::aligned(q.ptr, 16)) return fail(HINM_EALIGN, "%s: %s is not 16-byte aligned", whose, q.name);
  }
  return HINM_OK;
}

// The plan is every stack struct's first member.
int plan_of(const char* whose, const void* stack, const hinm_plan_t*& p) {
  if (!stack) return fail(HINM_EINVAL, "%s is NULL", whose);
  p = static_cast<const hinm_plan_t*>(stack);
  return hinm::check_plan(p);
}

template <int VALUES>
void launch(const MoeArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(moe_up_kernel<VALUES>, dim3(kCus), dim3(kThreads), 0, stream, a);
  hipLaunchKernelGGL(moe_down_kernel<VALUES>, dim3(kCus), dim3(kThreads), 0, stream, a);
}

}  // namespace

extern "C" int hinm_moe_layer_workspace_bytes(const hinm_plan_t* up, const hinm_plan_t* down, int32_t n_experts,
                                              int64_t n_tokens, int32_t top_k, size_t* bytes) {
  hinm::clear_error();
  int st = hinm::check_plan(up);
  if (st == HINM_OK) st = hinm::check_plan(down);
  if (st == HINM_OK) st = check_shapes(*up, *down, n_experts, n_tokens, top_k);
  if (st) return st;
  if (!bytes) return fail(HINM_EINVAL, "bytes is NULL");
  *bytes = (size_t)workspace_of(up->cin, up->cout, n_experts, n_tokens, top_k).bytes;
  return HINM_OK;
}

extern "C" int hinm_moe_layer(const void* logits, int32_t logits_type, int64_t ldl, const void* x_bf16,
                              int64_t n_tokens, int64_t ldx, int32_t n_experts, int32_t top_k, int32_t renormalize,
                              int32_t values, const void* gate, const void* up, const void* down, void* y_bf16,
                              int64_t ldy, void* workspace, size_t workspace_bytes, void* stream_) {
  hinm::clear_error();
  if (values != HINM_VALUES_BF16 && values != HINM_VALUES_MX4 && values != HINM_VALUES_FP8)
    return fail(HINM_EINVAL, "values=%d is none of HINM_VALUES_*", values);
  if (logits_type != HINM_BF16 && logits_type != HINM_FP32)
    return fail(HINM_EINVAL, "logits_type=%d is neither HINM_BF16 nor HINM_FP32", logits_type);
  const hinm_plan_t *pg, *pu, *pd;
  int st = plan_of("gate", gate, pg);
  if (st == HINM_OK) st = plan_of("up", up, pu);
  if (st == HINM_OK) st = plan_of("down", down, pd);
  if (st) return st;
  if (pg->cout != pu->cout || pg->cin != pu->cin || pg->tile_rows != pu->tile_rows)
    return fail(HINM_ESHAPE, "gate and up must have equal cout, cin and tile_rows");
  st = check_shapes(*pg, *pd, n_experts, n_tokens, top_k);
  if (st == HINM_OK) st = check_shapes(*pu, *pd, n_experts, n_tokens, top_k);
  if (st) return st;
  if (ldl < n_tokens || ldx < n_tokens || ldy < n_tokens)
    return fail(HINM_ESHAPE, "ldl=%lld, ldx=%lld and ldy=%lld must be >= the %lld tokens", (long long)ldl, (long long)ldx,
                (long long)ldy, (long long)n_tokens);
  if (n_tokens == 0) return HINM_OK;
  if (!logits || !x_bf16 || !y_bf16) return fail(HINM_EINVAL, "logits, x and y must be non-NULL");
  if (!hinm::aligned(logits, logits_type == HINM_FP32 ? 4 : 2) || !hinm::aligned(x_bf16, 2) || !hinm::aligned(y_bf16, 2))
    return fail(HINM_EALIGN, "logits, x and y must be aligned to their elements");
  MoeArgs a{};
  st = stack_of("gate", *pg, values, gate, a.gate);
  if (st == HINM_OK) st = stack_of("up", *pu, values, up, a.up);
  if (st == HINM_OK) st = stack_of("down", *pd, values, down, a.down);
  if (st) return st;
  const Workspace w = workspace_of(pu->cin, pu->cout, n_experts, n_tokens, top_k);
  if (!workspace || workspace_bytes < (size_t)w.bytes)
    return fail(HINM_EWORKSPACE, "workspace of %zu bytes given, %lld needed", workspace_bytes, (long long)w.bytes);
  if (!hinm::aligned(workspace, 256)) return fail(HINM_EALIGN, "workspace is not 256-byte aligned");
  st = hinm::ensure_device();
  if (st) return st;
  char* const ws = static_cast<char*>(workspace);
  a.logits = logits;
  a.logits_fp32 = logits_type == HINM_FP32;
  a.ldl = ldl;
  a.x = static_cast<const uint16_t*>(x_bf16);
  a.ldx = ldx;
  a.y = static_cast<uint16_t*>(y_bf16);
  a.ldy = ldy;
  a.table = reinterpret_cast<Table*>(ws + w.table);
  a.h = reinterpret_cast<uint16_t*>(ws + w.h);
  a.h_seg = w.h_seg;
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.counters = reinterpret_cast<unsigned*>(ws);
  a.n_tokens = (int)n_tokens;
  a.n_experts = n_experts;
  a.top_k = top_k;
  a.renormalize = renormalize != 0;
  a.up_cap = columns_of(pu->cin);
  a.down_cap = columns_of(pu->cout) / 2;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  if (values == HINM_VALUES_BF16) launch<HINM_VALUES_BF16>(a, stream);
  else if (values == HINM_VALUES_MX4) launch<HINM_VALUES_MX4>(a, stream);
  else launch<HINM_VALUES_FP8>(a, stream);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? HINM_OK : fail(HINM_EHIP, "mixture-of-experts layer's launch: %s", hipGetErrorString(e));
}
