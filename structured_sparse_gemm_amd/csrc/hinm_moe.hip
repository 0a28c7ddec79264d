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
constexpr int kMaxChannels = 16384;                // of four tokens, with the row of zeros
static_assert((kMaxChannels + 1) * 8 <= kSlab, "four tokens of the most channels fit");

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

// What the up kernel leaves for the down kernel.
struct Table {
  int n_seg;
  Seg seg[kPairs];
  uint16_t token[kPairs];          // by slot
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

// One K-block's operands of a lane: 64 rows' fragments f = 0 .. 3.
template <int VALUES>
struct Operand {                   // bf16
  u32x4 v[4];
  uint32_t m[4];
};
template <>
struct Operand<HINM_VALUES_MX4> {
  u32x4 v;
  uint32_t scale, m[2];
};
template <>
struct Operand<HINM_VALUES_FP8> {
  u32x2 v[4];
  uint32_t m[4], scale[4];
};

// acc += 64 rows (row block rb of the stack's rows) x 16 tokens over K-blocks
// v, v + nw, ... below b1, counted from b0; the activations are in `slab`,
// rows of `pitch` bytes, zeros in row cin.
template <int VALUES>
__device__ inline void multiply(const MoeStack& w, int expert, int rb, int b0, int b1, int v, int nw,
                                const uint8_t* slab, int pitch, f32x4 (&acc)[4]) {
  constexpr int D = 2;                             // blocks in flight
  const int lane = threadIdx.x & 63, i16 = lane & 15, kc = lane >> 4;
  const int nrb = w.rows / 64, t = rb / nrb, rt = rb % nrb;
  const __amdgpu_buffer_rsrc_t rvd = buffer(w.val_d + expert * w.b_val_d, w.b_val_d);
  const __amdgpu_buffer_rsrc_t rvs = buffer(w.val_s + expert * w.b_val_s, w.b_val_s);
  const __amdgpu_buffer_rsrc_t rm = buffer(w.meta + expert * w.b_meta, w.b_meta);
  const __amdgpu_buffer_rsrc_t rid = buffer(w.idx_d + expert * w.b_idx_d, w.b_idx_d);
  const __amdgpu_buffer_rsrc_t ris = buffer(w.idx_s + expert * w.b_idx_s, w.b_idx_s);
  const __amdgpu_buffer_rsrc_t rsd = buffer(w.scale_d + expert * w.b_scale_d, w.b_scale_d);
  const __amdgpu_buffer_rsrc_t rss = buffer(w.scale_s + expert * w.b_scale_s, w.b_scale_s);
  const int first = b0 + v, cnt = first < b1 ? (b1 - first + nw - 1) / nw : 0;
  if (cnt == 0) return;

  // Past the end the last block is read again, so that the loop has no
  // conditions; its products are not added.
  auto block = [&](int i) { return first + nw * min(i, cnt - 1); };
  auto load = [&](int i, Operand<VALUES>& o, int& iw) {
    const int b = block(i);
    const bool dense = b < w.nkb_d;
    const uint32_t k = (uint32_t)(dense ? b : b - w.nkb_d);
    const uint32_t kb = dense ? (uint32_t)(t * w.nkb_d) + k : (uint32_t)(t * w.nkb_s) + k;
    const __amdgpu_buffer_rsrc_t rv = dense ? rvd : rvs;
    iw = (int)__builtin_amdgcn_raw_buffer_load_b32(dense ? rid : ris, dense ? 4u * (lane & 31) : 4u * lane,
                                                   kb * (dense ? 128u : 256u), 0);
    if constexpr (VALUES == HINM_VALUES_MX4) {
      const uint32_t u = kb * (uint32_t)nrb + rt;
      o.v = __builtin_amdgcn_raw_buffer_load_b128(rv, 256u * kc + 16u * i16, u * 1024u, 0);
      o.scale = __builtin_amdgcn_raw_buffer_load_b32(dense ? rsd : rss, 4u * i16, u * 64u, 0);
      const u32x2 m = __builtin_amdgcn_raw_buffer_load_b64(rm, 128u * kc + 8u * i16, dense ? 0u : u * 512u, 0);
      o.m[0] = m[0];
      o.m[1] = m[1];
    } else {
      const uint32_t row = kb * (uint32_t)w.rows + rt * 64u;
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        if constexpr (VALUES == HINM_VALUES_FP8) {
          o.v[f] = __builtin_amdgcn_raw_buffer_load_b64(rv, 32u * i16 + 8u * kc + 512u * f, row * 32u, 0);
          const uint32_t group = dense ? (uint32_t)(t * ((w.nkb_d + 3) / 4)) + k / 4 : (uint32_t)(t * ((w.nkb_s + 3) / 4)) + k / 4;
          o.scale[f] = __builtin_amdgcn_raw_buffer_load_b8(dense ? rsd : rss, 16u * f + i16, group * w.rows + rt * 64u, 0);
        } else {
          o.v[f] = __builtin_amdgcn_raw_buffer_load_b128(rv, 64u * i16 + 16u * kc + 1024u * f, row * 64u, 0);
        }
        o.m[f] = __builtin_amdgcn_raw_buffer_load_b16(rm, 8u * i16 + 2u * kc + 128u * f, dense ? 0u : row * 8u, 0);
      }
    }
  };
  // The lane's share of the transposed reads: 8 bytes of tokens 4 s .. 4 s + 3
  // (past a short row the first ones again: columns that nothing reads) of
  // positions 8 kc + i16 / 4 + {0, 4, 32, 36}.
  const int s8 = 8 * min(i16 & 3, pitch / 8 - 1), p0 = 8 * kc + (i16 >> 2);
  auto compute = [&](int i, const Operand<VALUES>& o, int iw) {
    const bool dense = block(i) < w.nkb_d;
    const int row = (iw < 0 || iw >= w.cin ? w.cin : iw) * pitch;
    v4i16 b[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int p = p0 + 4 * (k & 1) + 32 * (k >> 1);
      // a dense block is multiplied as a 2:4 block whose groups keep positions 0 and 1: column 2 q + u at 4 q + u
      b[k] = tr_read_b(slab + __shfl(row, dense ? 2 * (p >> 2) + (p & 1) : p) + s8);
    }
    const bf16x8 lo8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7));
    const bf16x8 hi8 = __builtin_bit_cast(bf16x8, __builtin_shufflevector(b[2], b[3], 0, 1, 2, 3, 4, 5, 6, 7));
    const bf16x16 bv = __builtin_shufflevector(lo8, hi8, 0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
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
  };
  Operand<VALUES> o[D];
  int iw[D];
#pragma unroll
  for (int k = 0; k < D; ++k) load(k, o[k], iw[k]);
  for (int i = 0; i < cnt; i += D) {
#pragma unroll
    for (int k = 0; k < D; ++k) {
      if (i + k < cnt) compute(i + k, o[k], iw[k]);
      load(i + k + D, o[k], iw[k]);
    }
  }
}

// The wave's sums of fragment f into its 1 KiB: element (row r, token c) at 16 r + c.
__device__ inline void put_sums(float* red, const f32x4& acc) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int q = 0; q < 4; ++q) red[wave * 256 + (4 * (lane >> 4) + q) * 16 + (lane & 15)] = acc[q];
}

// ---------------------------------------------------------------------------
// Routing of all tokens, by every workgroup for itself (16 waves, a token at a
// time each: some 1 us, against a launch of its own).
// ---------------------------------------------------------------------------
struct RouteScratch {
  uint32_t mask[HINM_MAX_EXPERTS];       // tokens of every expert
  uint16_t start[HINM_MAX_EXPERTS];      // its first slot
  int16_t id[kPairs];
  float weight[kPairs];
};

__device__ inline float logit(const MoeArgs& a, int e, int n) {
  const float l = a.logits_fp32 ? static_cast<const float*>(a.logits)[e * a.ldl + n]
                                : __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[e * a.ldl + n] << 16);
  return l == l ? l : -__builtin_inff();
}

// The up kernel's segments and their tokens by slot go to `seg` and `token`;
// down (one workgroup's): the table for the down kernel.  Returns the number of
// segments through n_seg.
__device__ inline void route_tokens(const MoeArgs& a, RouteScratch& r, int* n_seg, Seg* seg, uint16_t* token, Table* down) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float none = -__builtin_inff();
  for (int e = threadIdx.x; e < a.n_experts; e += kThreads) r.mask[e] = 0u;
  __syncthreads();
  for (int n = wave; n < a.n_tokens; n += kWaves) {
    constexpr int kLane = HINM_MAX_EXPERTS / 64;
    float l[kLane];                                // experts lane + 64 i
#pragma unroll
    for (int i = 0; i < kLane; ++i) l[i] = 64 * i + lane < a.n_experts ? logit(a, 64 * i + lane, n) : none;
    float top = none, sum = 0.f, mine = 0.f;       // mine: lane j's exp(l_j - top)
    int chosen = -1;                               // lane j's expert
    for (int j = 0; j < a.top_k; ++j) {
      float best = none;
      int id = HINM_MAX_EXPERTS;
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (l[i] > best) best = l[i], id = 64 * i + lane;
      for (int d = 1; d < 64; d *= 2) {
        const float ob = __shfl_xor(best, d);
        const int oi = __shfl_xor(id, d);
        if (ob > best || (ob == best && oi < id)) best = ob, id = oi;
      }
      if (best == none) break;
      if (j == 0) {
        top = best;
        if (!a.renormalize) {
#pragma unroll
          for (int i = 0; i < kLane; ++i) sum += l[i] == top ? 1.f : l[i] == none ? 0.f : expf(l[i] - top);
          for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
        }
      }
      const float p = best == top ? 1.f : expf(best - top);
      if (a.renormalize) sum += p;
      if (lane == j) mine = p, chosen = id;
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (64 * i + lane == id) l[i] = none;
    }
    if (lane < a.top_k) {
      r.id[n * a.top_k + lane] = (int16_t)chosen;
      r.weight[n * a.top_k + lane] = chosen >= 0 ? mine / sum : 0.f;
      if (chosen >= 0) atomicOr(&r.mask[chosen], 1u << n);
    }
  }
  __syncthreads();
  // slots by expert and token, and the segments of both kernels
  if (wave == 0) {
    int slots = 0, ups = 0, downs = 0;             // of the experts before
    for (int e0 = 0; e0 < a.n_experts; e0 += 64) {
      const int e = e0 + lane;
      const int c = e < a.n_experts ? __popc(r.mask[e]) : 0;
      const int nu = (c + a.up_cap - 1) / a.up_cap, nd = (c + a.down_cap - 1) / a.down_cap;
      int sc = c, su = nu, sd = nd;
      for (int d = 1; d < 64; d *= 2) {
        const int vc = __shfl_up(sc, d), vu = __shfl_up(su, d), vd = __shfl_up(sd, d);
        if (lane >= d) sc += vc, su += vu, sd += vd;
      }
      const int s0 = slots + sc - c, u0 = ups + su - nu, d0 = downs + sd - nd;
      if (e < a.n_experts) r.start[e] = (uint16_t)s0;
      for (int q = 0; q < nu; ++q)
        seg[u0 + q] = {(uint16_t)e, (uint16_t)(s0 + q * a.up_cap), (uint8_t)min(a.up_cap, c - q * a.up_cap),
                          (uint8_t)(q * a.up_cap), (uint8_t)c, 0, (uint16_t)d0};
      if (down)
        for (int q = 0; q < nd; ++q)
          down->seg[d0 + q] = {(uint16_t)e, (uint16_t)(s0 + q * a.down_cap), (uint8_t)min(a.down_cap, c - q * a.down_cap),
                               (uint8_t)(q * a.down_cap), (uint8_t)c, 0, (uint16_t)d0};
      slots += __shfl(sc, 63);
      ups += __shfl(su, 63);
      downs += __shfl(sd, 63);
    }
    if (lane == 0) {
      *n_seg = ups;
      if (down) down->n_seg = downs;
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

template <int VALUES>
__global__ __launch_bounds__(kThreads) void moe_up_kernel(MoeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t slab[kSlab];
  __shared__ __attribute__((aligned(16))) union {
    float red[kWaves * 256];
    RouteScratch route;
  } sh;
  __shared__ int n_seg;
  __shared__ Seg segs[kPairs];
  __shared__ uint16_t token[kPairs];
  route_tokens(a, sh.route, &n_seg, segs, token, blockIdx.x == 0 ? a.table : nullptr);

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_rb = a.up.cout / 64;
  const int64_t items = (int64_t)n_seg * n_rb;
  const int i0 = (int)(blockIdx.x * items / gridDim.x), i1 = (int)((blockIdx.x + 1) * items / gridDim.x);
  const MoeStack& w = wave < kWaves / 2 ? a.gate : a.up;
  int held = -1, pitch = 8;
  for (int item = i0; item < i1; ++item) {
    const int sg = item / n_rb, rb = item % n_rb;
    const Seg seg = segs[sg];
    if (sg != held) {
      __syncthreads();
      pitch = 2 * row_columns(seg.n);
      for (int q = threadIdx.x; q < a.up.cin * (pitch / 2); q += kThreads) {
        const int c = q / (pitch / 2), j = q % (pitch / 2);
        reinterpret_cast<uint16_t*>(slab)[q] = j < seg.n ? a.x[c * a.ldx + token[seg.slot + j]] : (uint16_t)0;
      }
      if ((int)threadIdx.x < pitch / 2) reinterpret_cast<uint16_t*>(slab)[a.up.cin * (pitch / 2) + threadIdx.x] = 0;
      __syncthreads();
      held = sg;
    }
    f32x4 acc[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
    multiply<VALUES>(w, seg.expert, rb, 0, w.nkb_d + w.nkb_s, wave % (kWaves / 2), kWaves / 2, slab, pitch, acc);
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      put_sums(sh.red, acc[f]);
      __syncthreads();
      if (threadIdx.x < 256) {
        float g = 0.f, u = 0.f;
        for (int k = 0; k < kWaves / 2; ++k) {
          g += sh.red[k * 256 + threadIdx.x];
          u += sh.red[(kWaves / 2 + k) * 256 + threadIdx.x];
        }
        const int row = rb * 64 + 16 * f + (threadIdx.x >> 4), col = threadIdx.x & 15;
        if (col < seg.n) {
          // where the down kernel's segment of this token has it
          const int rank = seg.rank0 + col, q = rank / a.down_cap;
          const int width = row_columns(2 * min(a.down_cap, seg.count - q * a.down_cap));
          const float h = g / (1.f + expf(-g)) * u;
          const uint16_t hi = to_bf16(h);
          uint16_t* dst = a.h + (seg.down + q) * a.h_seg + (int64_t)row * width + rank % a.down_cap;
          dst[0] = hi;
          dst[width / 2] = to_bf16(h - __uint_as_float((uint32_t)hi << 16));
        }
      }
      __syncthreads();
    }
  }
}

template <int VALUES>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t slab[kSlab];
  __shared__ float red[kWaves * 256];
  __shared__ float out[64 * kTokens];
  __shared__ int s_last;
  const Table& table = *a.table;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_rb = a.down.cout / 64, nblk = a.down.nkb_d + a.down.nkb_s, n_seg = table.n_seg;
  const int units = n_seg * nblk;
  // shares of a row block's K-blocks: as many as leave no compute unit idle, and a block for each wave
  const int splits = max(1, min((int)gridDim.x / n_rb, units / kWaves));
  for (int item = blockIdx.x; item < n_rb * splits; item += gridDim.x) {
    const int rb = item / splits, split = item % splits;
    // whole segments in turn (an expert's are adjacent: they share its weights in the caches), then an even share of
    // the remaining ones' blocks
    const int rounds = n_seg / splits, rest = n_seg % splits * nblk, r0 = rounds * splits * nblk;
    const int u0 = r0 + (int)((int64_t)split * rest / splits), u1 = r0 + (int)((int64_t)(split + 1) * rest / splits);
    for (int q = threadIdx.x; q < 64 * kTokens; q += kThreads) out[q] = 0.f;
    for (int round = 0, u = u0; round < rounds || u < u1; ++round) {
      int sg = round * splits + split, b0 = 0, b1 = nblk;
      if (round >= rounds) {
        sg = u / nblk;
        b0 = u % nblk;
        b1 = min(nblk, b0 + u1 - u);
        u += b1 - b0;
      }
      const Seg seg = table.seg[sg];
      const int pitch = 2 * row_columns(2 * seg.n);
      __syncthreads();
      const u32x2* src = reinterpret_cast<const u32x2*>(a.h + sg * a.h_seg);
      for (int q = threadIdx.x; q < (a.down.cin + 1) * (pitch / 8); q += kThreads)
        reinterpret_cast<u32x2*>(slab)[q] = q < a.down.cin * (pitch / 8) ? src[q] : u32x2{0u, 0u};
      __syncthreads();
      f32x4 acc[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[f] = f32x4{0.f, 0.f, 0.f, 0.f};
      multiply<VALUES>(a.down, seg.expert, rb, b0, b1, wave, kWaves, slab, pitch, acc);
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        put_sums(red, acc[f]);
        __syncthreads();
        if (threadIdx.x < 256) {
          float s = 0.f;
          const int row = 16 * f + (threadIdx.x >> 4), col = threadIdx.x & 15, low = min(col + pitch / 4, 15) - col;
          for (int k = 0; k < kWaves; ++k) s += red[k * 256 + threadIdx.x] + red[k * 256 + threadIdx.x + low];
          if (col < seg.n) out[row * kTokens + table.token[seg.slot + col]] += table.weight[seg.slot + col] * s;
        }
        __syncthreads();
      }
    }
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
        for (int s = 0; s < splits; ++s)
#pragma unroll
          for (int k = 0; k < N; ++k)
            v[k] += __hip_atomic_load(p0 + (int64_t)s * 64 * kTokens + k * kThreads, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    if (last)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int q = k * kThreads + threadIdx.x, row = q / kTokens, n = q % kTokens;
        if (n < a.n_tokens) a.y[((int64_t)rb * 64 + row) * a.ldy + n] = to_bf16(v[k]);
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
