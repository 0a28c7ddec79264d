// Mixture-of-experts routing on [channels][tokens] activations: top-k experts
// and the column order by expert (hinm_route), token columns into that order
// (hinm_dispatch) and back (hinm_combine).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <climits>

#include "hinm_device.h"
#include "hinm_internal.h"

using hinm::fail;

namespace {

// ---------------------------------------------------------------------------
// Router.  Tokens are cut into blocks of kTok; a counting sort by expert needs
// three facts per (token, choice): the expert's first column (a prefix sum
// over the experts' totals), the choices of that expert in earlier blocks,
// and those of earlier tokens in the same block.  topk_kernel finds the
// choices and every block's expert counts, scan_kernel turns the counts into
// the counts of the blocks before (a column of them per expert) and the
// experts' totals, and place_kernel writes the order.  Up to kTok tokens, one
// workgroup does it all in one launch.
//
// The bytes are few (5 MB for 8192 tokens x 128 experts, 1 us): the three
// launches are bound by latency and by topk_kernel's compares, k per logit.
// 8192 x 128 fp32, top 8: 14.5 + 4.6 + 5.0 us; 16 tokens x 8 experts, top 2,
// in one launch: 4.8 us, about the time of an empty kernel.
// ---------------------------------------------------------------------------
constexpr int kTok = 64;           // tokens of a block: one wave's lanes
constexpr int kRouteThreads = 256;
constexpr int kScanExperts = 64;   // experts of a workgroup of scan_kernel: a wave's lanes
constexpr int kScanParts = 16;     // its waves, each a run of blocks

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  int n_tokens, n_experts, top_k, renormalize, align, bf16;
  int32_t *ids, *slots, *starts, *counts, *src;
  float* weights;
  int64_t n_cols;
  int n_blocks;
  int32_t *hist, *total;           // [n_blocks][n_experts], [n_experts]
};

// C logits of token n, experts e .. e1 - 1; -inf past e1, for a NaN and where
// `live` is false.  The loads themselves are unconditional (clamped), so that
// all of them are in flight at once.
template <int C>
__device__ inline void load_logits(const RouteArgs& a, int e, int e1, int n, bool live, float (&l)[C]) {
  const int nc = live ? n : 0;
  if (a.bf16) {
    const uint16_t* p = static_cast<const uint16_t*>(a.logits) + nc;
#pragma unroll
    for (int u = 0; u < C; ++u) l[u] = __uint_as_float((uint32_t)p[(int64_t)min(e + u, e1 - 1) * a.ldl] << 16);
  } else {
    const float* p = static_cast<const float*>(a.logits) + nc;
#pragma unroll
    for (int u = 0; u < C; ++u) l[u] = p[(int64_t)min(e + u, e1 - 1) * a.ldl];
  }
#pragma unroll
  for (int u = 0; u < C; ++u) l[u] = live && e + u < e1 && l[u] == l[u] ? l[u] : -INFINITY;
}

// A list of the K largest logits so far, descending, equal ones in the order
// they came in; -1 marks an empty place (no -inf logit enters).
template <int K>
struct Best {
  float v[K];
  int id[K];
  __device__ inline void clear() {
#pragma unroll
    for (int j = 0; j < K; ++j) {
      v[j] = -INFINITY;
      id[j] = -1;
    }
  }
  __device__ inline void add(float l, int e) {
    if (!(l > v[K - 1])) return;
    bool down = false;                           // once one entry moves, all after it do
#pragma unroll
    for (int j = 0; j < K; ++j) {
      down = down || l > v[j];
      const float tv = v[j];
      const int ti = id[j];
      v[j] = down ? l : tv;
      id[j] = down ? e : ti;
      l = down ? tv : l;
      e = down ? ti : e;
    }
  }
};

// Shared memory of the router's kernels, by phase.
template <int K>
struct RouteShared {
  union {
    struct {                                     // waves' lists and partial sums
      float v[4][K][kTok];
      int id[4][K][kTok];
    };
    unsigned long long mask[HINM_MAX_EXPERTS];   // per expert: the block's tokens that chose it
  };
  double sum[4][kTok];
  float top[kTok];
  int hist[HINM_MAX_EXPERTS];                    // the block's counts
  int before[HINM_MAX_EXPERTS];                  // counts of earlier blocks, then the block's first column
  int total[HINM_MAX_EXPERTS];
  int start[HINM_MAX_EXPERTS + 1];
  int part[4];                                   // waves' padded counts
};

// Choices and weights of tokens b * kTok ..; their experts' counts in s.hist.
// The four waves take a quarter of the experts each, one token a lane, and
// the first wave merges the four lists (in expert order, so equal logits stay
// in it).  Each thread ends up with its token's choices in the first wave.
// C: logits a thread holds at once (all of its quarter when that is no more).
template <int K, int C>
__device__ inline void topk_block(const RouteArgs& a, RouteShared<K>& s, int b, Best<K>& best) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = b * kTok + lane;
  const bool live = n < a.n_tokens;
  const int per = (a.n_experts + 3) / 4;
  // no tokens: nothing to read (logits may then be NULL); else lanes past the batch read token 0
  const int e0 = min(wave * per, a.n_experts), e1 = a.n_tokens > 0 ? min(e0 + per, a.n_experts) : e0;
  for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads) s.hist[e] = 0;
  best.clear();
  float l[C];
  for (int e = e0; e < e1; e += C) {
    load_logits<C>(a, e, e1, n, live, l);
#pragma unroll
    for (int u = 0; u < C; ++u) best.add(l[u], e + u);
  }
  // merge the four lists in two rounds: 1 into 0 and 3 into 2, then 2 into 0
  // (equal logits stay in expert order)
#pragma unroll
  for (int d = 1; d <= 2; d *= 2) {
    if (wave % (2 * d) == d) {
#pragma unroll
      for (int j = 0; j < K; ++j) {
        s.v[wave][j][lane] = best.v[j];
        s.id[wave][j][lane] = best.id[j];
      }
    }
    __syncthreads();
    if (wave % (2 * d) == 0) {
      float v[K];
      int id[K];
#pragma unroll
      for (int j = 0; j < K; ++j) {
        v[j] = s.v[wave + d][j][lane];
        id[j] = s.id[wave + d][j][lane];
      }
#pragma unroll
      for (int j = 0; j < K; ++j) best.add(v[j], id[j]);
    }
  }
  if (wave == 0) s.top[lane] = best.v[0];
  __syncthreads();
  // exp(l - m), where l == m gives 1 also for infinities.  The sum over all
  // experts is kept in 64 bits: up to 1024 terms, added one by one.
  const float m = s.top[lane];
  auto term = [&](float v) { return v == m ? 1.f : expf(v - m); };
  if (!a.renormalize) {
    double sum = 0.0;
    if (m > -INFINITY)
      for (int e = e0; e < e1; e += C) {
        if (per > C) load_logits<C>(a, e, e1, n, live, l);   // else l still holds them
#pragma unroll
        for (int u = 0; u < C; ++u)
          sum += l[u] > -INFINITY ? (double)term(l[u]) : 0.0;
      }
    s.sum[wave][lane] = sum;
    __syncthreads();
  }
  if (wave == 0 && live) {
    double sum = 0.0;
    if (a.renormalize) {
#pragma unroll
      for (int j = 0; j < K; ++j)
        if (j < a.top_k && best.id[j] >= 0) sum += (double)term(best.v[j]);
    } else {
      sum = s.sum[0][lane] + s.sum[1][lane] + s.sum[2][lane] + s.sum[3][lane];
    }
    const double inv = 1.0 / sum;
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < a.top_k) {
        const int e = best.id[j];
        a.ids[(int64_t)n * a.top_k + j] = e;
        a.weights[(int64_t)n * a.top_k + j] = e >= 0 ? (float)((double)term(best.v[j]) * inv) : 0.f;
        if (e >= 0) atomicAdd(&s.hist[e], 1);    // whole numbers: the order does not matter
      }
  }
  __syncthreads();
}

// First columns: s.start from the totals, and s.before, the counts of earlier
// blocks, becomes the block's own first column of every expert.
template <int K>
__device__ inline void scan_experts(const RouteArgs& a, RouteShared<K>& s) {
  // exclusive prefix sum of the padded totals: each thread a run of experts
  const int per = (a.n_experts + kRouteThreads - 1) / kRouteThreads;
  const int e0 = min((int)threadIdx.x * per, a.n_experts), e1 = min(e0 + per, a.n_experts);
  const int mask = a.align - 1, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int run = 0;
  for (int e = e0; e < e1; ++e) run += (s.total[e] + mask) & ~mask;
  int sum = run;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int v = __shfl_up(sum, d);
    sum += lane >= d ? v : 0;
  }
  if (lane == 63) s.part[wave] = sum;
  __syncthreads();
  int at = sum - run;
  for (int w = 0; w < wave; ++w) at += s.part[w];
  for (int e = e0; e < e1; ++e) {
    s.start[e] = at;
    s.before[e] += at;
    at += (s.total[e] + mask) & ~mask;
  }
  if (threadIdx.x == kRouteThreads - 1) s.start[a.n_experts] = at;
  __syncthreads();
}

// The order of block b's choices (ids of lane's token in `id`, -1 past the
// batch), and this block's share of the table of ranges and of the columns
// without a token.  s.before holds the first column of every expert for this
// block.
template <int K>
__device__ inline void place_block(const RouteArgs& a, RouteShared<K>& s, int b, const int (&id)[K]) {
  const int lane = threadIdx.x & 63;
  const int n = b * kTok + lane;
  for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads) s.mask[e] = 0ull;
  __syncthreads();
  if (threadIdx.x < 64) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < a.top_k && id[j] >= 0) atomicOr(&s.mask[id[j]], 1ull << lane);
  }
  __syncthreads();
  if (threadIdx.x < 64 && n < a.n_tokens) {
#pragma unroll
    for (int j = 0; j < K; ++j)
      if (j < a.top_k) {
        int slot = -1;
        if (id[j] >= 0) {
          slot = s.before[id[j]] + __popcll(s.mask[id[j]] & ((1ull << lane) - 1ull));
          if (slot < a.n_cols) a.src[slot] = n;  // always, given the columns the host asked for
        }
        a.slots[(int64_t)n * a.top_k + j] = slot;
      }
  }
  if (b == 0)
    for (int e = threadIdx.x; e <= a.n_experts; e += kRouteThreads) {
      a.starts[e] = s.start[e];
      if (e < a.n_experts) a.counts[e] = s.total[e];
    }
  for (int e = b; e < a.n_experts; e += a.n_blocks)
    for (int64_t c = s.start[e] + s.total[e] + threadIdx.x; c < min((int64_t)s.start[e + 1], a.n_cols);
         c += kRouteThreads)
      a.src[c] = -1;
  for (int64_t c = s.start[a.n_experts] + (int64_t)b * kRouteThreads + threadIdx.x; c < a.n_cols;
       c += (int64_t)a.n_blocks * kRouteThreads)
    a.src[c] = -1;
}

template <int K, int C, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void topk_kernel(RouteArgs a) {
  __shared__ RouteShared<K> s;
  Best<K> best;
  topk_block<K, C>(a, s, blockIdx.x, best);
  if constexpr (ONE) {
    for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads) {
      s.total[e] = s.hist[e];
      s.before[e] = 0;
    }
    __syncthreads();
    scan_experts<K>(a, s);
    const bool live = (int)threadIdx.x < a.n_tokens;
#pragma unroll
    for (int j = 0; j < K; ++j) best.id[j] = live ? best.id[j] : -1;
    place_block<K>(a, s, 0, best.id);
  } else {
    for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads)
      a.hist[(int64_t)blockIdx.x * a.n_experts + e] = s.hist[e];
  }
}

// Counts of every block -> counts of the blocks before it, and the totals: a
// lane an expert, a wave a run of blocks.
__global__ __launch_bounds__(kScanParts * 64) void scan_kernel(RouteArgs a) {
  __shared__ int part[kScanParts][kScanExperts];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * kScanExperts + lane;
  const int per = (a.n_blocks + kScanParts - 1) / kScanParts;
  const int b0 = min(wave * per, a.n_blocks), b1 = min(b0 + per, a.n_blocks);
  const bool live = e < a.n_experts;
  int32_t* col = a.hist + (live ? e : 0);
  constexpr int U = 8;                           // loads in flight
  int sum = 0;
  for (int b = b0; b < b1; b += U) {
    int v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = b + u < b1 ? col[(int64_t)(b + u) * a.n_experts] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) sum += v[u];
  }
  part[wave][lane] = sum;
  __syncthreads();
  int at = 0;
  for (int w = 0; w < wave; ++w) at += part[w][lane];
  if (wave == kScanParts - 1 && live) a.total[e] = at + sum;
  for (int b = b0; b < b1; b += U) {
    int v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = b + u < b1 ? col[(int64_t)(b + u) * a.n_experts] : 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u < b1 && live) col[(int64_t)(b + u) * a.n_experts] = at;
      at += v[u];
    }
  }
}

template <int K>
__global__ __launch_bounds__(kRouteThreads) void place_kernel(RouteArgs a) {
  __shared__ RouteShared<K> s;
  const int b = blockIdx.x, lane = threadIdx.x & 63, n = b * kTok + lane;
  int id[K];
#pragma unroll
  for (int j = 0; j < K; ++j)
    id[j] = threadIdx.x < 64 && n < a.n_tokens && j < a.top_k ? a.ids[(int64_t)n * a.top_k + j] : -1;
  for (int e = threadIdx.x; e < a.n_experts; e += kRouteThreads) {
    s.total[e] = a.total[e];
    s.before[e] = a.hist[(int64_t)b * a.n_experts + e];
  }
  __syncthreads();
  scan_experts<K>(a, s);
  place_block<K>(a, s, b, id);
}

// ---------------------------------------------------------------------------
// Dispatch and combine: bound by the bytes of the two matrices.  A column's
// source may be anywhere in a row, and 2-byte gathers from memory run at a
// quarter of the copy rate, so a workgroup stages G whole rows in LDS,
// interleaved (a token's G values are one LDS word of 2 G bytes), and one LDS
// read brings G rows of a column.  G is the largest of 8, 4, 2, 1 whose rows
// fit 80 KB (two workgroups a compute unit); longer rows are gathered from
// memory.  4096 rows, 4096 tokens x 2 choices: dispatch 21 us, combine 28 us
// (101 MB each, 4.8 and 3.6 TB/s; gathered from memory 39 and 68 us).
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 512;
constexpr int kMoveLds = 80 * 1024;
constexpr int64_t kMoveWgs = 1024;
constexpr int64_t kMoveMax = 1 << 30;  // columns and tokens: a thread's next one still fits an int
constexpr int kMoveRows = 16;      // channels a workgroup of the direct kernels walks

typedef u32x4 any_u32x4 __attribute__((aligned(2)));   // 16 bytes at any 2-byte aligned address
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 any_u32x2 __attribute__((aligned(2)));

template <int G>
struct Rows;                       // a token's values of G rows
template <>
struct Rows<8> { u32x4 w; };
template <>
struct Rows<4> { u32x2 w; };
template <>
struct Rows<2> { uint32_t w[1]; };
template <>
struct Rows<1> { uint16_t w[1]; };

// Halves of two words: both low (hi = 0) or both high halves, a's first.
__device__ inline uint32_t pair(uint32_t a, uint32_t b, int hi) {
  return __builtin_amdgcn_perm(b, a, hi ? 0x07060302u : 0x05040100u);
}

// Eight tokens' rows as G rows of eight tokens.
template <int G>
__device__ inline void to_rows(const Rows<G> (&t)[8], u32x4 (&v)[G]) {
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int r = 0; r < G; ++r) v[r][u] = pair(t[2 * u].w[r / 2], t[2 * u + 1].w[r / 2], r & 1);
}

// Rows c0 .. c0 + G - 1 of a matrix into LDS (rows past `channels` as zeros).
// A thread brings two adjacent tokens at a time, so that a wave's LDS stores
// are contiguous, and four such pairs before it stores any.
template <int G>
__device__ inline void stage_rows(const uint16_t* __restrict__ x, int64_t ldx, int n, int64_t c0, int64_t channels,
                                  Rows<G>* buf) {
  typedef uint32_t any_u32 __attribute__((aligned(2)));
  constexpr int P = 4;
  for (int q0 = threadIdx.x * 2; q0 < n; q0 += kMoveThreads * 2 * P) {
    uint32_t v[P][G];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int q = q0 + p * kMoveThreads * 2;
#pragma unroll
      for (int r = 0; r < G; ++r) {
        v[p][r] = 0u;
        if (q < n && c0 + r < channels) {
          const uint16_t* src = x + (c0 + r) * ldx + q;
          v[p][r] = q + 1 < n ? *reinterpret_cast<const any_u32*>(src) : (uint32_t)*src;
        }
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int q = q0 + p * kMoveThreads * 2;
      Rows<G> t[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if constexpr (G == 1) t[u].w[0] = (uint16_t)(v[p][0] >> (16 * u));
        else
#pragma unroll
          for (int k = 0; k < G / 2; ++k) t[u].w[k] = pair(v[p][2 * k], v[p][2 * k + 1], u);
      }
      if (q < n) {                               // an odd row's last pair: its second half is never read
        buf[q] = t[0];
        buf[q + 1] = t[1];
      }
    }
  }
}

template <int G>
__global__ __launch_bounds__(kMoveThreads) void dispatch_kernel(const uint16_t* __restrict__ x, int64_t channels,
                                                                int n_tokens, int64_t ldx,
                                                                const int32_t* __restrict__ src, int n_cols,
                                                                uint16_t* __restrict__ xs, int64_t ldxs) {
  __shared__ __attribute__((aligned(16))) Rows<G> buf[kMoveLds / (2 * G)];
  for (int64_t c0 = (int64_t)blockIdx.x * G; c0 < channels; c0 += (int64_t)gridDim.x * G) {
    stage_rows<G>(x, ldx, n_tokens, c0, channels, buf);
    __syncthreads();
    for (int col = threadIdx.x * 8; col < n_cols; col += kMoveThreads * 8) {
      const int left = n_cols - col;
      Rows<G> t[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int s = u < left ? src[col + u] : -1;
        t[u] = Rows<G>{};
        if (s >= 0 && s < n_tokens) t[u] = buf[s];
      }
      u32x4 v[G];
      to_rows<G>(t, v);
#pragma unroll
      for (int r = 0; r < G; ++r)
        if (c0 + r < channels) {
          uint16_t* dst = xs + (c0 + r) * ldxs + col;
          if (left >= 8) *reinterpret_cast<any_u32x4*>(dst) = v[r];
          else
            for (int u = 0; u < 8; ++u)
              if (u < left) dst[u] = (uint16_t)(v[r][u >> 1] >> (16 * (u & 1)));
        }
    }
    __syncthreads();
  }
}

// Four tokens a thread; every token's sum runs over its choices in order.  K:
// top_k when it is 1 or 2 (a thread's slots and weights then are whole 16-byte
// words), 0 for any other.
template <int G, int K>
__global__ __launch_bounds__(kMoveThreads) void combine_kernel(const uint16_t* __restrict__ ys, int64_t channels,
                                                               int n_cols, int64_t ldys,
                                                               const int32_t* __restrict__ slots,
                                                               const float* __restrict__ weights, int n_tokens,
                                                               int top_k, uint16_t* __restrict__ y, int64_t ldy) {
  __shared__ __attribute__((aligned(16))) Rows<G> buf[kMoveLds / (2 * G)];
  for (int64_t c0 = (int64_t)blockIdx.x * G; c0 < channels; c0 += (int64_t)gridDim.x * G) {
    stage_rows<G>(ys, ldys, n_cols, c0, channels, buf);
    __syncthreads();
    for (int n = threadIdx.x * 4; n < n_tokens; n += kMoveThreads * 4) {
      const int left = n_tokens - n;
      float acc[4][G];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < G; ++r) acc[u][r] = 0.f;
      auto add = [&](int u, int s, float w) {
        if (s >= 0 && s < n_cols) {
          const Rows<G> t = buf[s];
#pragma unroll
          for (int r = 0; r < G; ++r) {
            const uint32_t h = t.w[r / 2];
            acc[u][r] = fmaf(w, __uint_as_float(r & 1 ? h & 0xffff0000u : h << 16), acc[u][r]);
          }
        }
      };
      if (K > 0 && left >= 4) {
        typedef u32x4 word_u32x4 __attribute__((aligned(4)));
        u32x4 s[K ? K : 1], w[K ? K : 1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          s[k] = *reinterpret_cast<const word_u32x4*>(slots + (int64_t)n * K + 4 * k);
          w[k] = *reinterpret_cast<const word_u32x4*>(weights + (int64_t)n * K + 4 * k);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < K; ++j)
            add(u, (int)s[(u * K + j) / 4][(u * K + j) % 4], __uint_as_float(w[(u * K + j) / 4][(u * K + j) % 4]));
      } else {
        for (int j = 0; j < top_k; ++j)
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (u < left) add(u, slots[(int64_t)(n + u) * top_k + j], weights[(int64_t)(n + u) * top_k + j]);
      }
#pragma unroll
      for (int r = 0; r < G; ++r)
        if (c0 + r < channels) {
          uint16_t* dst = y + (c0 + r) * ldy + n;
          uint16_t h[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) h[u] = bf16_rne(acc[u][r]);
          if (left >= 4) *reinterpret_cast<any_u32x2*>(dst) = u32x2{h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16)};
          else
            for (int u = 0; u < 4; ++u)
              if (u < left) dst[u] = h[u];
        }
    }
    __syncthreads();
  }
}

// Rows too long for LDS: gathered from memory, a thread walking channels with
// its columns' sources in registers.
__global__ __launch_bounds__(256) void dispatch_direct_kernel(const uint16_t* __restrict__ x, int64_t channels,
                                                              int n_tokens, int64_t ldx,
                                                              const int32_t* __restrict__ src, int n_cols,
                                                              uint16_t* __restrict__ xs, int64_t ldxs) {
  const int64_t col = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (col >= n_cols) return;
  const int left = (int)min((int64_t)8, n_cols - col);
  int t[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) t[u] = u < left ? src[col + u] : -1;
  for (int64_t c0 = (int64_t)blockIdx.y * kMoveRows; c0 < channels; c0 += (int64_t)gridDim.y * kMoveRows)
    for (int64_t c = c0; c < min(c0 + kMoveRows, channels); ++c) {
      u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (t[u] >= 0 && t[u] < n_tokens) v[u >> 1] |= (uint32_t)x[c * ldx + t[u]] << (16 * (u & 1));
      uint16_t* dst = xs + c * ldxs + col;
      if (left == 8) *reinterpret_cast<any_u32x4*>(dst) = v;
      else
        for (int u = 0; u < left; ++u) dst[u] = (uint16_t)(v[u >> 1] >> (16 * (u & 1)));
    }
}

__global__ __launch_bounds__(256) void combine_direct_kernel(const uint16_t* __restrict__ ys, int64_t channels,
                                                             int n_cols, int64_t ldys,
                                                             const int32_t* __restrict__ slots,
                                                             const float* __restrict__ weights, int n_tokens,
                                                             int top_k, uint16_t* __restrict__ y, int64_t ldy) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= n_tokens) return;
  for (int64_t c0 = (int64_t)blockIdx.y * kMoveRows; c0 < channels; c0 += (int64_t)gridDim.y * kMoveRows)
    for (int64_t c = c0; c < min(c0 + kMoveRows, channels); ++c) {
      float acc = 0.f;
      for (int j = 0; j < top_k; ++j) {
        const int s = slots[(int64_t)n * top_k + j];
        if (s >= 0 && s < n_cols)
          acc = fmaf(weights[(int64_t)n * top_k + j], __uint_as_float((uint32_t)ys[c * ldys + s] << 16), acc);
      }
      y[c * ldy + n] = bf16_rne(acc);
    }
}

// Rows a workgroup stages for a row of n elements; 0: they do not fit.
int staged_rows(int64_t n) {
  for (int g = 8; g; g /= 2)
    if ((n + 1) * 2 * g <= kMoveLds) return g;   // pairs of elements: one more than an odd row has
  return 0;
}

int launch_status(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? HINM_OK : fail(HINM_EHIP, "%s launch: %s", what, hipGetErrorString(e));
}

int check_router(int64_t n_tokens, int32_t n_experts) {
  if (n_tokens < 0) return fail(HINM_ESHAPE, "n_tokens=%lld is negative", (long long)n_tokens);
  if (n_experts < 1 || n_experts > HINM_MAX_EXPERTS)
    return fail(HINM_ESHAPE, "n_experts=%d; 1 to %d are supported", n_experts, HINM_MAX_EXPERTS);
  if (n_tokens > (1 << 26)) return fail(HINM_ESHAPE, "n_tokens=%lld exceeds 2^26", (long long)n_tokens);
  return HINM_OK;
}

int check_choice(int64_t n_tokens, int32_t n_experts, int32_t top_k, int32_t align) {
  const int st = check_router(n_tokens, n_experts);
  if (st) return st;
  if (top_k < 1 || top_k > n_experts || top_k > HINM_MAX_TOP_K)
    return fail(HINM_ESHAPE, "top_k=%d; 1 to min(n_experts=%d, %d) are supported", top_k, n_experts, HINM_MAX_TOP_K);
  if (align < 1 || align > HINM_MAX_ALIGN || (align & (align - 1)))
    return fail(HINM_EINVAL, "align=%d is not a power of two up to %d", align, HINM_MAX_ALIGN);
  return HINM_OK;
}

int64_t route_columns(int64_t n_tokens, int32_t n_experts, int32_t top_k, int32_t align) {
  const int64_t used = n_tokens * top_k;
  return (used + std::min<int64_t>(n_experts, used) * (align - 1) + align - 1) / align * align;
}

// [counts of every block][totals]
void route_shape(int64_t n_tokens, int32_t n_experts, int* n_blocks, size_t* bytes) {
  *n_blocks = (int)std::max<int64_t>(1, (n_tokens + kTok - 1) / kTok);
  *bytes = *n_blocks == 1 ? 0 : (size_t)(*n_blocks + 1) * n_experts * sizeof(int32_t);
}

template <int K, int C>
int launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.n_blocks == 1) {
    hipLaunchKernelGGL((topk_kernel<K, C, true>), dim3(1), dim3(kRouteThreads), 0, stream, a);
    return launch_status("route");
  }
  hipLaunchKernelGGL((topk_kernel<K, C, false>), dim3(a.n_blocks), dim3(kRouteThreads), 0, stream, a);
  int st = launch_status("route");
  if (st) return st;
  hipLaunchKernelGGL(scan_kernel, dim3((a.n_experts + kScanExperts - 1) / kScanExperts), dim3(kScanParts * 64), 0, stream, a);
  st = launch_status("route");
  if (st) return st;
  hipLaunchKernelGGL(place_kernel<K>, dim3(a.n_blocks), dim3(kRouteThreads), 0, stream, a);
  return launch_status("route");
}

// Logits a thread holds: its quarter of 8, 32 or 128 experts.
template <int K>
int launch_route(const RouteArgs& a, hipStream_t stream) {
  if constexpr (K <= 8)                          // 16 choices need more than 8 experts
    if (a.n_experts <= 8) return launch_route<K, 2>(a, stream);
  if (a.n_experts <= 32) return launch_route<K, 8>(a, stream);
  return launch_route<K, 32>(a, stream);
}

}  // namespace

extern "C" int hinm_route_columns(int64_t n_tokens, int32_t n_experts, int32_t top_k, int32_t align,
                                  int64_t* n_cols) {
  hinm::clear_error();
  const int st = check_choice(n_tokens, n_experts, top_k, align);
  if (st) return st;
  if (!n_cols) return fail(HINM_EINVAL, "n_cols is NULL");
  *n_cols = route_columns(n_tokens, n_experts, top_k, align);
  return HINM_OK;
}

extern "C" int hinm_route_workspace_bytes(int64_t n_tokens, int32_t n_experts, size_t* bytes) {
  hinm::clear_error();
  const int st = check_router(n_tokens, n_experts);
  if (st) return st;
  if (!bytes) return fail(HINM_EINVAL, "bytes is NULL");
  int nb;
  route_shape(n_tokens, n_experts, &nb, bytes);
  return HINM_OK;
}

extern "C" int hinm_route(const void* logits, int32_t logits_type, int64_t n_tokens, int64_t ldl, int32_t n_experts,
                          int32_t top_k, int32_t renormalize, int32_t align, int32_t* ids, float* weights,
                          int32_t* slots, int32_t* starts, int32_t* counts, int32_t* src, int64_t n_cols,
                          void* workspace, size_t workspace_bytes, void* stream_) {
  hinm::clear_error();
  int st = check_choice(n_tokens, n_experts, top_k, align);
  if (st) return st;
  if (logits_type != HINM_BF16 && logits_type != HINM_FP32)
    return fail(HINM_EINVAL, "logits_type=%d is neither HINM_BF16 nor HINM_FP32", logits_type);
  if (ldl < n_tokens) return fail(HINM_ESHAPE, "ldl=%lld is below n_tokens=%lld", (long long)ldl, (long long)n_tokens);
  const int64_t need = route_columns(n_tokens, n_experts, top_k, align);
  if (n_cols < need)
    return fail(HINM_ESHAPE, "n_cols=%lld, this routing needs %lld", (long long)n_cols, (long long)need);
  if (n_cols > INT32_MAX) return fail(HINM_ESHAPE, "n_cols=%lld does not fit in int32", (long long)n_cols);
  if (!starts || !counts || (n_cols > 0 && !src) || (n_tokens > 0 && (!logits || !ids || !weights || !slots)))
    return fail(HINM_EINVAL, "logits and the outputs must be non-NULL");
  if (!hinm::aligned(logits, logits_type == HINM_BF16 ? 2 : 4)) return fail(HINM_EALIGN, "logits is misaligned");
  for (const void* p : {(const void*)ids, (const void*)weights, (const void*)slots, (const void*)starts,
                        (const void*)counts, (const void*)src})
    if (!hinm::aligned(p, 4)) return fail(HINM_EALIGN, "the outputs must be 4-byte aligned");
  RouteArgs a;
  size_t bytes;
  route_shape(n_tokens, n_experts, &a.n_blocks, &bytes);
  if (bytes > 0) {
    if (!workspace || workspace_bytes < bytes)
      return fail(HINM_EWORKSPACE, "route workspace of %zu bytes given, %zu needed", workspace_bytes, bytes);
    if (!hinm::aligned(workspace, 256)) return fail(HINM_EALIGN, "workspace is not 256-byte aligned");
  }
  st = hinm::ensure_device();
  if (st) return st;
  a.logits = logits;
  a.ldl = ldl;
  a.n_tokens = (int)n_tokens;
  a.n_experts = n_experts;
  a.top_k = top_k;
  a.renormalize = renormalize != 0;
  a.align = align;
  a.bf16 = logits_type == HINM_BF16;
  a.ids = ids;
  a.weights = weights;
  a.slots = slots;
  a.starts = starts;
  a.counts = counts;
  a.src = src;
  a.n_cols = n_cols;
  a.hist = static_cast<int32_t*>(workspace);
  a.total = a.hist ? a.hist + (size_t)a.n_blocks * n_experts : nullptr;
  hipStream_t stream = reinterpret_cast<hipStream_t>(stream_);
  const hinm::EnqueueLock whole(workspace);
  if (top_k == 1) return launch_route<1>(a, stream);
  if (top_k == 2) return launch_route<2>(a, stream);
  if (top_k <= 4) return launch_route<4>(a, stream);
  if (top_k <= 8) return launch_route<8>(a, stream);
  return launch_route<16>(a, stream);
}

extern "C" int hinm_dispatch(const void* x_bf16, int64_t channels, int64_t n_tokens, int64_t ldx, const int32_t* src,
                             int64_t n_cols, void* xs_bf16, int64_t ldxs, void* stream) {
  hinm::clear_error();
  if (channels < 0 || n_tokens < 0 || n_cols < 0)
    return fail(HINM_ESHAPE, "channels, n_tokens and n_cols must not be negative");
  if (channels > INT32_MAX || n_tokens > kMoveMax || n_cols > kMoveMax)
    return fail(HINM_ESHAPE, "channels must be below 2^31, n_tokens and n_cols at most 2^30");
  if (ldx < n_tokens || ldxs < n_cols)
    return fail(HINM_ESHAPE, "ldx=%lld must be >= n_tokens=%lld and ldxs=%lld >= n_cols=%lld", (long long)ldx,
                (long long)n_tokens, (long long)ldxs, (long long)n_cols);
  if (channels == 0 || n_cols == 0) return HINM_OK;
  if (!src || !xs_bf16 || (n_tokens > 0 && !x_bf16)) return fail(HINM_EINVAL, "x, src and xs must be non-NULL");
  if (!hinm::aligned(x_bf16, 2) || !hinm::aligned(xs_bf16, 2) || !hinm::aligned(src, 4))
    return fail(HINM_EALIGN, "x and xs must be 2-byte aligned, src 4-byte aligned");
  const int st = hinm::ensure_device();
  if (st) return st;
  hipStream_t st_ = reinterpret_cast<hipStream_t>(stream);
  const uint16_t* x = static_cast<const uint16_t*>(x_bf16);
  uint16_t* xs = static_cast<uint16_t*>(xs_bf16);
  const int nt = (int)n_tokens, nc = (int)n_cols, g = staged_rows(n_tokens);
  if (g) {
    const dim3 grid((unsigned)std::min<int64_t>((channels + g - 1) / g, kMoveWgs)), block(kMoveThreads);
    switch (g) {
      case 8: hipLaunchKernelGGL(dispatch_kernel<8>, grid, block, 0, st_, x, channels, nt, ldx, src, nc, xs, ldxs); break;
      case 4: hipLaunchKernelGGL(dispatch_kernel<4>, grid, block, 0, st_, x, channels, nt, ldx, src, nc, xs, ldxs); break;
      case 2: hipLaunchKernelGGL(dispatch_kernel<2>, grid, block, 0, st_, x, channels, nt, ldx, src, nc, xs, ldxs); break;
      default: hipLaunchKernelGGL(dispatch_kernel<1>, grid, block, 0, st_, x, channels, nt, ldx, src, nc, xs, ldxs); break;
    }
  } else {
    const dim3 grid((unsigned)((n_cols + 2047) / 2048),
                    (unsigned)std::min<int64_t>((channels + kMoveRows - 1) / kMoveRows, 65535));
    hipLaunchKernelGGL(dispatch_direct_kernel, grid, dim3(256), 0, st_, x, channels, nt, ldx, src, nc, xs, ldxs);
  }
  return launch_status("dispatch");
}

extern "C" int hinm_combine(const void* ys_bf16, int64_t channels, int64_t n_cols, int64_t ldys, const int32_t* slots,
                            const float* weights, int64_t n_tokens, int32_t top_k, void* y_bf16, int64_t ldy,
                            void* stream) {
  hinm::clear_error();
  if (channels < 0 || n_tokens < 0 || n_cols < 0)
    return fail(HINM_ESHAPE, "channels, n_tokens and n_cols must not be negative");
  if (channels > INT32_MAX || n_tokens > kMoveMax || n_cols > kMoveMax)
    return fail(HINM_ESHAPE, "channels must be below 2^31, n_tokens and n_cols at most 2^30");
  if (top_k < 1 || top_k > HINM_MAX_TOP_K) return fail(HINM_ESHAPE, "top_k=%d; 1 to %d are supported", top_k, HINM_MAX_TOP_K);
  if (ldy < n_tokens || ldys < n_cols)
    return fail(HINM_ESHAPE, "ldy=%lld must be >= n_tokens=%lld and ldys=%lld >= n_cols=%lld", (long long)ldy,
                (long long)n_tokens, (long long)ldys, (long long)n_cols);
  if (channels == 0 || n_tokens == 0) return HINM_OK;
  if (!slots || !weights || !y_bf16 || (n_cols > 0 && !ys_bf16))
    return fail(HINM_EINVAL, "ys, slots, weights and y must be non-NULL");
  if (!hinm::aligned(ys_bf16, 2) || !hinm::aligned(y_bf16, 2) || !hinm::aligned(slots, 4) || !hinm::aligned(weights, 4))
    return fail(HINM_EALIGN, "ys and y must be 2-byte aligned, slots and weights 4-byte aligned");
  const int st = hinm::ensure_device();
  if (st) return st;
  hipStream_t st_ = reinterpret_cast<hipStream_t>(stream);
  const uint16_t* ys = static_cast<const uint16_t*>(ys_bf16);
  uint16_t* y = static_cast<uint16_t*>(y_bf16);
  const int nt = (int)n_tokens, nc = (int)n_cols, g = staged_rows(n_cols);
  if (g) {
    const dim3 grid((unsigned)std::min<int64_t>((channels + g - 1) / g, kMoveWgs)), block(kMoveThreads);
#define HINM_COMBINE_K(G_, K_)                                                                                       \
  hipLaunchKernelGGL((combine_kernel<G_, K_>), grid, block, 0, st_, ys, channels, nc, ldys, slots, weights, nt, top_k, \
                     y, ldy)
#define HINM_COMBINE(G_)                                                                                             \
  do {                                                                                                               \
    if (top_k == 1) HINM_COMBINE_K(G_, 1);                                                                           \
    else if (top_k == 2) HINM_COMBINE_K(G_, 2);                                                                      \
    else HINM_COMBINE_K(G_, 0);                                                                                      \
  } while (0)
    switch (g) {
      case 8: HINM_COMBINE(8); break;
      case 4: HINM_COMBINE(4); break;
      case 2: HINM_COMBINE(2); break;
      default: HINM_COMBINE(1); break;
    }
#undef HINM_COMBINE
#undef HINM_COMBINE_K
  } else {
    const dim3 grid((unsigned)((n_tokens + 255) / 256),
                    (unsigned)std::min<int64_t>((channels + kMoveRows - 1) / kMoveRows, 65535));
    hipLaunchKernelGGL(combine_direct_kernel, grid, dim3(256), 0, st_, ys, channels, nc, ldys, slots, weights, nt,
                       top_k, y, ldy);
  }
  return launch_status("combine");
}
