// hinm_moe_layer: a gated mixture-of-experts layer for a few tokens in two
// kernels (formulas at hinm_moe_layer).
//
// A few tokens make a layer a read of the chosen experts' packed weights, so
// both kernels are built around that stream: every wave keeps its own K-blocks
// in flight.
//
//   up kernel    every workgroup works out the routing from the logits, then
//                takes (segment, 32 or 64 inner channels); a segment is
//                up to 16 of an expert's tokens.  Their activations are held in
//                LDS whole, [channel][token], and the channels that a tile
//                keeps gathered there: the transposed LDS read takes an address
//                a lane, which is the channel's row.  Four waves take the
//                gate's K-blocks, four the up projection's; the sums meet in
//                LDS and become h, which goes to the workspace by channels.
//   down kernel  a workgroup takes 64 rows of Y and a share of all segments'
//                K-blocks.  h has more channels than X and two columns a token,
//                too much for LDS, so a wave gathers a block's rows of h from
//                L2, by indices that it read a turn before, and turns them
//                through LDS of its own.  A segment's sums are multiplied by
//                the router's weights and added to the tokens' in LDS, and the
//                shares meet in the workspace.  (With h in LDS a segment held
//                two tokens of 11008 channels, and 8 experts of 8 tokens each
//                took 145 us, four reads of each expert's weight; now 75.)
//
// What bounds them (8 experts of 11008x4096, bf16, 32 tokens, 104 and 75 us for
// 418 and 209 MB): a compute unit's 64 outstanding cache lines, of which the
// gathered rows of h are most in the down kernel.  One token (26 and 19 us for
// 104 and 52 MB): a third is the chain ahead of the first products - arguments,
// logits, choices, the segments' list, first loads, each after the one before.
//
// h is a matrix operand and so bf16, but rounded once it would cost the output
// as much as its own rounding (relative error of the layer 0.0024, against
// 0.0017 from the rounding of Y alone).  It is held as the sum of two bf16
// values instead, its rounding and what that leaves, in two columns of the
// matrix instruction, of which a few tokens leave many idle.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "hinm_device.h"
#include "hinm_fp8.h"
#include "hinm_internal.h"
#include "hinm_mx4.h"
#include "hinm_ragged.h"
#include "hinm_stream.h"

using hinm::Buf;
using hinm::check_bufs;
using hinm::fail;

namespace {

constexpr int kWaves = 8;                          // of a workgroup; one workgroup a compute unit (16: slower)
constexpr int kThreads = 64 * kWaves;
constexpr int kTokens = HINM_MOE_MAX_TOKENS;
constexpr int kPairs = kTokens * HINM_MAX_TOP_K;   // (token, expert) pairs at most; a segment holds at least one
constexpr int kSlab = 131328;                      // bytes of LDS for a segment's activations and a row of zeros
constexpr int kMaxChannels = 16384;                // of four columns, with the row of zeros
static_assert((kMaxChannels + 1) * 8 <= kSlab, "four columns of the most channels fit");
// Floats between the waves' sums of F fragments, the 8 for reads free of bank conflicts.
constexpr int sums_pitch(int f) { return 256 * f + 8; }

// Reads a word of every 64 bytes of a kernel's arguments, so that they are in
// the scalar cache when they are wanted, and waited for once (a token, 2 of 8
// experts of 11008: 48.2 us without, 47.5 with).
template <class Args>
__device__ __forceinline__ void touch(const Args& a) {
  uint32_t x = 0;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Args) + 63) / 64; ++i) x ^= reinterpret_cast<const uint32_t*>(&a)[16 * i];
  asm volatile("" ::"s"(x));
}

// One stack of packed weights; strides are bytes of one expert.
struct MoeStack {
  const uint8_t *val_d, *val_s, *scale_d, *scale_s, *meta, *idx_d, *idx_s;
  int64_t b_val_d, b_val_s, b_scale_d, b_scale_s, b_meta, b_idx_d, b_idx_s;
  int rows, nkb_d, nkb_s, cin, cout;
};

// A segment: n of an expert's tokens, from the rank0-th on.
struct Seg {
  uint32_t mask;                   // the tokens
  uint16_t expert, down;           // down: the expert's first segment of the down kernel
  uint8_t n, rank0;
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
  uint16_t* h;                     // [segment][inner channels and a row of zeros][wide]
  float* part;
  unsigned* counters;
  int64_t ldl, ldx, ldy, h_seg;    // h_seg: elements between segments
  int logits_fp32, n_tokens, n_experts, top_k, renormalize, up_cap, wide;   // wide: twice a segment's tokens there
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

__device__ inline Source source_of(const MoeStack& w, const Item& it, int v) {
  const int t = (unsigned)(it.rows16 * 16) / (unsigned)w.rows;
  const int64_t e = it.expert;
  return {w.val_d + e * w.b_val_d, w.val_s + e * w.b_val_s, w.meta + e * w.b_meta, w.idx_d + e * w.b_idx_d,
          w.idx_s + e * w.b_idx_s, w.scale_d + e * w.b_scale_d, w.scale_s + e * w.b_scale_s,
          t, it.rows16 * 16 - t * w.rows, it.b0 + v, it.b1};
}

// The index of block b's position p (of a dense block's 32, twice).
__device__ inline int load_index(const MoeStack& w, const Source& s, int b, uint32_t p) {
  const bool dense = b < w.nkb_d;
  const uint32_t kb = dense ? s.tile * w.nkb_d + b : s.tile * w.nkb_s + b - w.nkb_d;
  return at<int>(pick(dense, s.idx_d, s.idx_s), dense ? kb * 128 + 4 * (p & 31) : kb * 256 + 4 * p);
}

// Block b's operands.  The block's place is scalar and the lane's share a
// constant; a dense block has no metadata and reads its values' bytes instead.
template <int VALUES, int F>
__device__ inline void load_block(const MoeStack& w, const Source& s, int b, Operand<VALUES, F>& o) {
  const uint32_t lane = threadIdx.x & 63, i16 = lane & 15, kc = lane >> 4;
  const bool dense = b < w.nkb_d;
  const uint32_t k = dense ? b : b - w.nkb_d, nkb = dense ? w.nkb_d : w.nkb_s, kb = s.tile * nkb + k;   // offsets below 2^31
  const uint8_t *val = pick(dense, s.val_d, s.val_s), *scale = pick(dense, s.scale_d, s.scale_s), *meta = pick(dense, val, s.meta);
  if constexpr (VALUES == HINM_VALUES_MX4) {
    const uint32_t u = kb * (w.rows / 64) + s.row / 64;
    const uint32_t f0 = (uint32_t)(s.row >> 4) & 3;          // 0 or 2 with two fragments
    o.scale = at<uint32_t>(scale, u * 64 + 4 * i16) >> (8 * f0);
    if constexpr (F == 4) {
      const u32x4 v = at<u32x4>(val, u * 1024 + 256 * kc + 16 * i16);
      const u32x2 m = at<u32x2>(meta, u * 512 + 128 * kc + 8 * i16);
      for (int f = 0; f < 4; ++f) o.v[f] = v[f];
      o.m[0] = m[0];
      o.m[1] = m[1];
    } else {
      const u32x2 v = at<u32x2>(val, u * 1024 + 256 * kc + 16 * i16 + 4 * f0);
      o.v[0] = v[0];
      o.v[1] = v[1];
      o.m[0] = at<uint32_t>(meta, u * 512 + 128 * kc + 8 * i16 + 2 * f0);
    }
  } else {
    constexpr int kRow = VALUES == HINM_VALUES_FP8 ? 32 : 64;      // bytes of a row
    const uint32_t row = kb * w.rows + s.row, group = (s.tile * ((nkb + 3) / 4) + k / 4) * w.rows + s.row;
#pragma unroll
    for (int f = 0; f < F; ++f) {
      if constexpr (VALUES == HINM_VALUES_FP8) {
        o.v[f] = at<u32x2>(val, row * kRow + 32 * i16 + 8 * kc + 512 * f);
        o.scale[f] = at<uint8_t>(scale, group + 16 * f + i16);
      } else {
        o.v[f] = at<u32x4>(val, row * kRow + 64 * i16 + 16 * kc + 1024 * f);
      }
      o.m[f] = at<uint16_t>(meta, row * 8 + 8 * i16 + 2 * kc + 128 * f);
    }
  }
}

// acc += the block's rows x 16 columns, of which row(position) is the LDS row.
// The lane's share of the transposed reads: 8 bytes of columns 4 s .. 4 s + 3
// (past a short row the first ones again: columns that nothing reads) of
// positions 8 kc + i16 / 4 + {0, 4, 32, 36}.  A dense block is multiplied as a
// 2:4 block whose groups keep positions 0 and 1: column 2 q + u at 4 q + u.
template <int VALUES, int F, class Row>
__device__ inline void multiply_block(bool dense, const Operand<VALUES, F>& o, int pitch, Row row, f32x4 (&acc)[F]) {
  const int lane = threadIdx.x & 63, i16 = lane & 15, kc = lane >> 4;
  const int s8 = 8 * min(i16 & 3, pitch / 8 - 1), p0 = 8 * kc + (i16 >> 2);
  v4i16 q[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int p = p0 + 4 * (k & 1) + 32 * (k >> 1);
    q[k] = tr_read_b(row(dense ? 2 * (p >> 2) + (p & 1) : p) + s8);
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
// Of those broadcasts, lanes of the rows of 16 in ROWS alone.
template <int CTRL, int ROWS>
__device__ inline uint32_t to_row(uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xf, false); }
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
__device__ __forceinline__ void load_logits(const MoeArgs& a, int n, uint32_t (&raw)[NL]) {
  const int lane = threadIdx.x & 63;
  n = min(n, a.n_tokens - 1);
  if (a.logits_fp32) {
#pragma unroll
    for (int i = 0; i < NL; ++i) raw[i] = static_cast<const uint32_t*>(a.logits)[min(64 * i + lane, a.n_experts - 1) * a.ldl + n];
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) raw[i] = static_cast<const uint16_t*>(a.logits)[min(64 * i + lane, a.n_experts - 1) * a.ldl + n];
  }
}
template <int NL>
__device__ __forceinline__ void route_token(const MoeArgs& a, RouteScratch& r, int n, const uint32_t (&raw)[NL]) {
  const int lane = threadIdx.x & 63;
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

// The up kernel's segments go to `seg`, their number to n_seg; down (one
// workgroup's): the table for the down kernel.  meanwhile() runs while the
// first logits come.
template <class Meanwhile>
__device__ __forceinline__ void route_tokens(const MoeArgs& a, RouteScratch& r, int* n_seg, Seg* seg, Table* down, Meanwhile meanwhile) {
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), down_cap = a.wide / 2;
  for (int e = threadIdx.x; e < a.n_experts; e += kThreads) r.mask[e] = 0u;
  auto tokens = [&](auto count) {
    constexpr int NL = decltype(count)::value;
    uint32_t raw[NL];
    load_logits<NL>(a, wave, raw);
    meanwhile();
    step_barrier();                                // the masks are clear
    for (int n = wave; n < a.n_tokens; n += kWaves) {
      if (n != wave) load_logits<NL>(a, n, raw);
      route_token<NL>(a, r, n, raw);
    }
  };
  if (a.n_experts <= 64) tokens(std::integral_constant<int, 1>{});
  else if (a.n_experts <= 256) tokens(std::integral_constant<int, 4>{});
  else tokens(std::integral_constant<int, HINM_MAX_EXPERTS / 64>{});
  step_barrier();
  // slots by expert and token, and the segments of both kernels; the three running counts (each at most kPairs) share
  // a word
  if (wave == 0) {
    uint32_t before = 0;                           // counts of the experts before
#pragma nounroll
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < a.n_experts ? __popc(r.mask[e]) : 0;
      const int nu = (c + a.up_cap - 1) / a.up_cap, nd = (c + down_cap - 1) / down_cap;
      const uint32_t own = (uint32_t)c | (uint32_t)nu << 10 | (uint32_t)nd << 20;
      uint32_t all = own;                          // over the lanes up to this one
      all += shifted<0x111>(all);
      all += shifted<0x112>(all);
      all += shifted<0x114>(all);
      all += shifted<0x118>(all);
      all += to_row<0x142, 0xa>(all);
      all += to_row<0x143, 0xc>(all);
      const uint32_t at = before + all - own;
      const int s0 = at & 1023, u0 = at >> 10 & 1023, d0 = at >> 20;
      if (e < a.n_experts) r.start[e] = (uint16_t)s0;
      uint32_t rest = nu ? r.mask[e] : 0u;
      for (int q = 0; q < nu; ++q) {
        const int n = min(a.up_cap, c - q * a.up_cap);
        uint32_t after = rest;
        for (int j = 0; j < n; ++j) after &= after - 1u;
        seg[u0 + q] = {rest & ~after, (uint16_t)e, (uint16_t)d0, (uint8_t)n, (uint8_t)(q * a.up_cap)};
        rest = after;
      }
      if (down)
        for (int q = 0; q < nd; ++q)
          down->seg[d0 + q] = (uint32_t)e | (uint32_t)(s0 + q * down_cap) << 10 | (uint32_t)min(down_cap, c - q * down_cap) << 20;
      before += (uint32_t)__builtin_amdgcn_readlane((int)all, 63);
    }
    if (lane == 0) {
      *n_seg = before >> 10 & 1023;
      if (down) down->n_seg = before >> 20;
    }
  }
  step_barrier();
  if (down && (int)threadIdx.x < a.n_tokens * a.top_k) {
    const int e = r.id[threadIdx.x], n = threadIdx.x / a.top_k;
    if (e >= 0) {
      const int slot = r.start[e] + __popc(r.mask[e] & ((1u << n) - 1u));
      down->token[slot] = (uint16_t)n;
      down->weight[slot] = r.weight[threadIdx.x];
    }
  }
  step_barrier();
}

// X's values of eight tokens, g .. g + 7 (of fewer than eight the rows' first
// ones, and the last rows' loads begin early; where fewer follow g, the last
// eight), of channels c0 .. c0 + 8 * 512 - 1.
constexpr int kHeld = 8;
__device__ inline int first_token(const MoeArgs& a, int g) { return a.n_tokens < 8 ? 0 : min(g, a.n_tokens - 8); }
__device__ __forceinline__ void load_x(const MoeArgs& a, int g, int c0, u32x4 (&v)[kHeld]) {
  const int tid = own_thread();
  const uint16_t* const x = a.x + first_token(a, g);
  const int64_t last = a.n_tokens < 8 ? (int64_t)(a.up.cin - 1) * a.ldx + a.n_tokens - 8 : INT64_MAX;   // 64 elements or more
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const uint32_t c = min(c0 + tid + u * kThreads, a.up.cin - 1);
    v[u] = *reinterpret_cast<const any_u32x4*>(x + min((int64_t)((uint64_t)c * (uint32_t)a.ldx), last));
  }
}
// Those of the tokens `mask` into the slab, from column col on.
__device__ __forceinline__ void put_x(const MoeArgs& a, uint32_t mask, int g, int c0, int col, int width, u32x4 (&v)[kHeld],
                                      uint16_t* slab) {
  const int tid = own_thread();
  const uint32_t some = ((mask >> g) & 255u) << (g - first_token(a, g));
  uint16_t* at[kHeld];                             // past the last channel that one again, and its values
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const int c = min(c0 + tid + u * kThreads, a.up.cin - 1);
    at[u] = slab + c * width + col;
    if (a.n_tokens < 8) {
      const int64_t past = (int64_t)((uint64_t)(uint32_t)c * (uint32_t)a.ldx) - ((int64_t)(a.up.cin - 1) * a.ldx + a.n_tokens - 8);
      if (__ballot(past > 0)) v[u] = shifted_row(v[u], (int)max(past, (int64_t)0));
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t)
    if ((some >> t) & 1u) {
#pragma unroll
      for (int u = 0; u < kHeld; ++u) *at[u]++ = (uint16_t)(v[u][t >> 1] >> (16 * (t & 1)));
    }
}

// Items are (segment, 16 F rows of the inner channels).  A turn of three blocks: of
// two, three and four, a token's layer 49.0, 47.5 and 49.7 us (bf16), 41.9, 40.6
// and 42.0 (8 bits), 32 tokens 179, 176 and 179, 152, 149 and 153 (this and the
// figures below: three sets of inputs in turn).
template <int VALUES, int F>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
  constexpr int R = 16 * F, kPitch = sums_pitch(2), kDepth = 3;
  __shared__ __attribute__((aligned(16))) uint8_t slab[kSlab];
  __shared__ __attribute__((aligned(16))) union {
    float red[kWaves * kPitch];
    RouteScratch route;
  } sh;
  __shared__ int n_seg;
  __shared__ Seg segs[kPairs];
  touch(a);
  u32x4 v[kHeld];
  // the first loads of up to eight tokens' activations need no routing
  bool early = a.n_tokens <= 8;
  route_tokens(a, sh.route, &n_seg, segs, blockIdx.x == 0 ? a.table : nullptr, [&] {
    if (early) load_x(a, 0, 0, v);
  });

  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const unsigned n_rb = a.up.cout / R;
  const Share mine = share_of(uniform(n_seg), n_rb);               // at most 512 * 512 items
  const MoeStack& w = wave < kWaves / 2 ? a.gate : a.up;
  const int nd = w.nkb_d;
  int held = -1, coming = -1, rb = 0, pitch = 8;
  Seg seg{};                       // of the item at hand
  f32x4 acc[F];
  auto seg_at = [&](unsigned sg) -> Seg {
    const Seg t = segs[sg];
    return {(uint32_t)uniform(t.mask), (uint16_t)uniform(t.expert), (uint16_t)uniform(t.down), (uint8_t)uniform(t.n), (uint8_t)uniform(t.rank0)};
  };
  auto group_of = [](uint32_t mask) { return __builtin_ctz(mask) & ~7; };
  stream<Operand<VALUES, F>, Source, kDepth, kWaves / 2>(
      (int)mine.n,
      [&](int i) -> Source {
        const unsigned sg = (mine.first + i) / n_rb;
        const Seg next = seg_at(sg);
        if ((int)sg != coming) {
          coming = sg;
          if (!early) load_x(a, group_of(next.mask), 0, v);
          early = false;
        }
        return source_of(w, {next.expert, (int)(mine.first + i - sg * n_rb) * F, 0, nd + w.nkb_s}, wave % (kWaves / 2));
      },
      [&](const Source& s, int b, Operand<VALUES, F>& o) {
        o.index = load_index(w, s, b, lane);
        load_block<VALUES, F>(w, s, b, o);
      },
      [&](int b, const Operand<VALUES, F>& o) {
        const int row = ((uint32_t)o.index < (uint32_t)w.cin ? o.index : w.cin) * pitch;
        multiply_block<VALUES, F>(b < nd, o, pitch, [&](int p) { return slab + __shfl(row, p); }, acc);
      },
      [&](int i) {
        const unsigned sg = (mine.first + i) / n_rb;
        rb = mine.first + i - sg * n_rb;
        if ((int)sg != held) {
          held = sg;
          seg = seg_at(sg);
          const int width = row_columns(seg.n);
          pitch = 2 * width;
          uint32_t left = seg.mask;
          int col = 0, g = group_of(left);
#pragma nounroll
          for (int c0 = 0;;) {
            put_x(a, left, g, c0, col, width, v, reinterpret_cast<uint16_t*>(slab));
            c0 += kHeld * kThreads;
            if (c0 >= a.up.cin) {
              col += __popc((left >> g) & 255u);
              left &= ~(255u << g);
              if (!left) break;
              g = group_of(left);
              c0 = 0;
            }
            load_x(a, g, c0, v);
          }
          const int tid = own_thread();
          if (tid < width) reinterpret_cast<uint16_t*>(slab)[a.up.cin * width + tid] = 0;
          step_barrier();
        }
#pragma unroll
        for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
      },
      [&](int) {
        // two fragments at a time, which is what LDS has room for: a lane's sums of wave w, fragment f to
        // red[w][f % 2][lane]; of four adjacent threads the first two sum the gate's waves, the others the up
        // projection's, and each makes one row's h
#pragma unroll
        for (int f0 = 0; f0 < F; f0 += 2) {
#pragma unroll
          for (int f = 0; f < 2; ++f) *reinterpret_cast<f32x4*>(sh.red + wave * kPitch + 256 * f + 4 * lane) = acc[f0 + f];
          step_barrier();
          const int tid = own_thread(), part = tid & 3, t = tid >> 2;
          const f32x4 s = *reinterpret_cast<const f32x4*>(sh.red + 2 * part * kPitch + 4 * t) +
                          *reinterpret_cast<const f32x4*>(sh.red + (2 * part + 1) * kPitch + 4 * t);
          float own = 0.f, other = 0.f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float x = s[q] + quad1(s[q]), y = quad2(x);
            if (q == part) own = x, other = y;
          }
          const float g = part < 2 ? own : other, u = part < 2 ? other : own;
          const int col = t & 15, row = 16 * (f0 + (t >> 6)) + 4 * ((t >> 4) & 3) + part;
          if (col < seg.n) {
            // where the down kernel's segment of this token has it
            const int rank = seg.rank0 + col, cap = a.wide / 2, q = rank / cap;
            const float h = g / (1.f + expf(-g)) * u;
            const uint16_t hi = to_bf16(h);
            const float rest = h - __uint_as_float((uint32_t)hi << 16);
            uint16_t* const dst = a.h + (seg.down + q) * a.h_seg + rank - q * cap;
            uint16_t* const at = dst + (rb * R + row) * a.wide;
            at[0] = hi;
            at[cap] = to_bf16(fabsf(rest) < __builtin_inff() ? rest : 0.f);      // an infinite h stays infinite
            if (rb == 0 && row == 0) dst[a.up.cout * a.wide] = dst[a.up.cout * a.wide + cap] = 0;
          }
          step_barrier();
        }
      });
}

// A workgroup's K-blocks are a contiguous range of those of all segments, its
// items the parts of it in one segment.  In a turn of kDepth blocks a wave
// multiplies those whose rows and values it asked for a turn before, asks for
// the rows and values of the next ones, by indices that it asked for a turn
// before, and for the indices of those after.  No load is under a condition:
// waits are for a known number of loads.
// A turn of two blocks: of two, three and four, a token's layer 47.5, 48.4 and
// 50.4 us (bf16), 40.6, 41.6 and 43.5 (8 bits).
template <int VALUES, int WIDE>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
  constexpr int F = 4, kPitch = sums_pitch(F), kDepth = 2, kRow = 2 * WIDE, kSlot = 64 * kRow;
  typedef std::conditional_t<WIDE == 4, u32x2, u32x4> Piece;
  constexpr int kPieces = kRow / sizeof(Piece);    // of a row, which as many adjacent lanes read: they share a cache line
  __shared__ __attribute__((aligned(16))) uint8_t slots[kWaves * 2 * kSlot];
  __shared__ __attribute__((aligned(16))) float red[kWaves * kPitch];
  __shared__ float out[64 * kTokens];              // [row][token]
  __shared__ Table table;
  __shared__ int s_last;
  touch(a);
  const int wave = uniform(threadIdx.x >> 6), lane = threadIdx.x & 63;
  for (int q = threadIdx.x; q < (int)sizeof(Table) / 4; q += kThreads)
    reinterpret_cast<uint32_t*>(&table)[q] = reinterpret_cast<const uint32_t*>(a.table)[q];
  __syncthreads();
  const MoeStack& w = a.down;
  const int n_rb = w.cout / 64, nd = w.nkb_d, nblk = nd + w.nkb_s, n_seg = uniform(table.n_seg), units = n_seg * nblk;
  // shares of a row block's K-blocks: as many as one round of workgroups holds, with a block for each wave (of 256
  // workgroups all at 4096 hidden channels, 240 at 5120, 192 at 6144, 224 at 7168)
  const int splits = max(1, min(kCus / n_rb, units / kWaves));
  uint8_t* const slot = slots + wave * 2 * kSlot;
#pragma nounroll
  for (int item = blockIdx.x; item < n_rb * splits; item += kCus) {
    const int rb = item / splits, split = item % splits;
    const int u0 = split * units / splits, u1 = (split + 1) * units / splits;      // below 2^20 * splits
    const int s0 = n_seg ? u0 / nblk : 0, parts = u0 < u1 ? (u1 - 1) / nblk - s0 + 1 : 0;
    for (int q = threadIdx.x; q < 64 * a.n_tokens; q += kThreads) out[q] = 0.f;
    step_barrier();
    auto source = [&](int i) {
      const int sg = s0 + i;
      return source_of(w, {uniform(table.seg[sg] & 1023), rb * F, max(0, u0 - sg * nblk), min(nblk, u1 - sg * nblk)}, wave);
    };
    auto turns_of = [&](const Source& s) { return max(1, (s.end - s.first + kDepth * kWaves - 1) / (kDepth * kWaves)); };
    f32x4 acc[F];
#pragma unroll
    for (int f = 0; f < F; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto finish = [&](int i) {
      const int word = uniform((int)table.seg[s0 + i]), first = word >> 10 & 1023, n = word >> 20;
#pragma unroll
      for (int f = 0; f < F; ++f) *reinterpret_cast<f32x4*>(red + wave * kPitch + 256 * f + 4 * lane) = acc[f];
      step_barrier();
      const int tid = own_thread(), part = tid & 1, t = tid >> 1;    // four waves' sums of fragment t / 64, lane t % 64
      f32x4 s = *reinterpret_cast<const f32x4*>(red + 4 * part * kPitch + 4 * t);
#pragma unroll
      for (int k = 1; k < 4; ++k) s += *reinterpret_cast<const f32x4*>(red + (4 * part + k) * kPitch + 4 * t);
      const int col = t & 15, row = 16 * (t >> 6) + 4 * ((t >> 4) & 3);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x = s[q] + quad1(s[q]);
        x += __shfl_down(x, WIDE);                 // the token's other column, WIDE / 2 further on
        if ((q & 1) == part && col < n) out[(row + q) * a.n_tokens + table.token[first + col]] += table.weight[first + col] * x;
        acc[q] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      step_barrier();
    };
    if (parts > 0) {
      Operand<VALUES, F> o[kDepth];
      Piece rows[kDepth][kPieces];
      int index[kDepth][kPieces], asked[kDepth], block[kDepth];        // blocks; ~b: block b, not to be multiplied
      int seg_i = 0;                                         // the item that indices are asked of
      Source src = source(0), from;
      int turns = turns_of(src), ends = -1, last = -1;       // items that the turns of rows and of products end
      const uint8_t* h_src = reinterpret_cast<const uint8_t*>(a.h + s0 * a.h_seg);
      const uint8_t* h_from = h_src;
      auto ask = [&](int k) {
        const int b = min(src.first, src.end - 1);
#pragma unroll
        for (int u = 0; u < kPieces; ++u) index[k][u] = load_index(w, src, b, 64 / kPieces * u + lane / kPieces);
        asked[k] = src.first < src.end ? b : ~b;
        src.first += kWaves;
      };
      // ends the turn of indices: which item it ends, and on to the next one
      auto turn = [&] {
        from = src;
        h_from = h_src;
        ends = -1;
        if (--turns > 0) return;
        turns = 1;
        if (seg_i < parts) ends = seg_i;
        if (++seg_i < parts) {
          src = source(seg_i);
          turns = turns_of(src);
          h_src += 2 * a.h_seg;
        }
      };
#pragma unroll
      for (int k = 0; k < kDepth; ++k) {
        ask(k);
        block[k] = -1;
      }
      turn();
#pragma nounroll
      while (true) {
        const int ended = last;
        last = ends;
#pragma unroll
        for (int k = 0; k < kDepth; ++k) {
          if (block[k] >= 0) {
            uint8_t* const to = slot + (k & 1) * kSlot;
#pragma unroll
            for (int u = 0; u < kPieces; ++u) *reinterpret_cast<Piece*>(to + (64 * u + lane) * sizeof(Piece)) = rows[k][u];
            multiply_block<VALUES, F>(block[k] < nd, o[k], kRow, [&](int p) { return to + p * kRow; }, acc);
          }
          block[k] = asked[k];
          const int b = asked[k] < 0 ? ~asked[k] : asked[k];
#pragma unroll
          for (int u = 0; u < kPieces; ++u) {
            const uint32_t row = (uint32_t)index[k][u] < (uint32_t)w.cin ? index[k][u] : w.cin;
            rows[k][u] = at<Piece>(h_from, row * kRow + lane % kPieces * sizeof(Piece));
          }
          load_block<VALUES, F>(w, from, b, o[k]);
          ask(k);
        }
        turn();
        if (ended >= 0) {
          finish(ended);
          if (ended == parts - 1) break;
        }
      }
    }
    const int outs = 64 * a.n_tokens;
    bool leave = false;
    float* const part0 = a.part + (int64_t)rb * splits * 64 * kTokens;
    if (splits > 1) {
      float* const my = part0 + (int64_t)split * 64 * kTokens;
      for (int q = threadIdx.x; q < outs; q += kThreads) __hip_atomic_store(my + q, out[q], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      if (threadIdx.x == 0) s_last = arrive(a.counters + rb, splits);
      __syncthreads();
      leave = !s_last;
    }
    if (!leave)
      for (int q = threadIdx.x; q < outs; q += kThreads) {
        float v = splits > 1 ? 0.f : out[q];
        if (splits > 1)
#pragma unroll 4
          for (int s = 0; s < splits; ++s)
            v += __hip_atomic_load(part0 + (int64_t)s * 64 * kTokens + q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const unsigned row = (unsigned)q / (unsigned)a.n_tokens, col = q - row * a.n_tokens;
        a.y[((int64_t)rb * 64 + row) * a.ldy + col] = to_bf16(v);
      }
    __syncthreads();
  }
}

// Tokens that a segment of the up kernel holds at most: as many as fit in LDS.
int columns_of(int channels) { return (channels + 1) * 32 <= kSlab ? 16 : (channels + 1) * 16 <= kSlab ? 8 : 4; }

// Columns of h, twice the tokens of a segment of the down kernel: of 16 its
// products use what there is, but of up to two tokens rows of 8 bytes are fewer
// loads.
int wide_of(int64_t n_tokens) { return n_tokens <= 2 ? 4 : 16; }

struct Workspace {
  int64_t table, part, h, h_seg, bytes;            // offsets; h_seg in elements
};
Workspace workspace_of(int hidden, int inter, int32_t n_experts, int64_t n_tokens, int32_t top_k) {
  Workspace w{};
  if (n_tokens == 0) return w;
  const int64_t pairs = n_tokens * top_k, wide = wide_of(n_tokens);
  const int64_t segs = std::min(pairs, std::min<int64_t>(n_experts, pairs) + pairs / (wide / 2));
  w.table = hinm::kWsCounterBytes;
  w.part = w.table + (int64_t)((sizeof(Table) + 255) / 256 * 256);
  const int64_t items = std::max<int64_t>(kCus, hidden / 64);
  w.h = w.part + items * 64 * kTokens * 4;
  w.h_seg = (int64_t)(inter + 1) * wide;
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
  return check_bufs(b, 7, whose);
}

// The plan is every stack struct's first member.
int plan_of(const char* whose, const void* stack, const hinm_plan_t*& p) {
  if (!stack) return fail(HINM_EINVAL, "%s is NULL", whose);
  p = static_cast<const hinm_plan_t*>(stack);
  return hinm::check_plan(p);
}

// Fragments of 16 rows of the up kernel's items: what leaves the busiest
// workgroup the least to do, by an item's cost of its own, in half fragments.
// Measured with two and with four (8 experts of 11008x4096, top 2): bf16 at 1
// and 32 tokens 48 / 52 and 176 / 176 us, 8 bits 41 / 45 and 149 / 150, 4 bits
// 34 / 33 and 127 / 113.
int fragments_of(const MoeArgs& a, int values) {
  const int64_t segs = std::min<int64_t>(a.n_experts, (int64_t)a.n_tokens * a.top_k);
  const int own = values == HINM_VALUES_MX4 ? 6 : 0;
  auto cost = [&](int f) { return (segs * (a.up.cout / (16 * f)) + kCus - 1) / kCus * (2 * f + own); };
  return cost(2) <= cost(4) ? 2 : 4;
}

template <int VALUES>
void launch(const MoeArgs& a, hipStream_t stream) {
  if (fragments_of(a, VALUES) == 2) hipLaunchKernelGGL((moe_up_kernel<VALUES, 2>), dim3(kCus), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((moe_up_kernel<VALUES, 4>), dim3(kCus), dim3(kThreads), 0, stream, a);
  if (a.wide == 4) hipLaunchKernelGGL((moe_down_kernel<VALUES, 4>), dim3(kCus), dim3(kThreads), 0, stream, a);
  else hipLaunchKernelGGL((moe_down_kernel<VALUES, 16>), dim3(kCus), dim3(kThreads), 0, stream, a);
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
  if (ldx >= (int64_t)1 << 31) return fail(HINM_ESHAPE, "ldx=%lld must be below 2^31", (long long)ldx);
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
  a.wide = wide_of(n_tokens);
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  const hinm::EnqueueLock whole(workspace);
  if (values == HINM_VALUES_BF16) launch<HINM_VALUES_BF16>(a, stream);
  else if (values == HINM_VALUES_MX4) launch<HINM_VALUES_MX4>(a, stream);
  else launch<HINM_VALUES_FP8>(a, stream);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? HINM_OK : fail(HINM_EHIP, "mixture-of-experts layer's launch: %s", hipGetErrorString(e));
}
