// The loop of the kernels for a few tokens (not installed): a wave's share of
// the K-blocks of several items, as one stream of loads.
#ifndef HINM_STREAM_H_
#define HINM_STREAM_H_

#include "hinm_device.h"
#include "hinm_ragged.h"

namespace {

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// A barrier that waits for this wave's LDS operations, not for its loads.
__device__ inline void step_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The thread's number, as a value that the compiler takes for new: what is
// computed from it stays where it is used, and out of the code ahead of a loop
// that uses it once.
__device__ inline int own_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

template <class T>
__device__ inline T at(const uint8_t* base, uint32_t offset) { return *reinterpret_cast<const T*>(base + offset); }

// a or b, both evaluated: a choice between two members in place would become
// one between their addresses, and put the struct on the stack.
__device__ inline const uint8_t* pick(bool c, const uint8_t* a, const uint8_t* b) { return c ? a : b; }

// While DEPTH of a wave's blocks are multiplied the next DEPTH blocks' operands
// are on their way, across the items' ends too.  For item i:
//   open(i)       names the wave's blocks, first, first + NW, ... below end, and
//                 where they lie (the item has one block at least, for some
//                 wave), and where the item begins a segment asks for its
//                 activations, ahead of the weight;
//   load(s, b, o) loads block b's operands;
//   multiply(b, o) adds its products;
//   begin(i), finish(i): before its first and after its last product, in step
//                 for the whole workgroup.
// One loop body serves the first loads, the products and the items' ends.  The
// weight's loads are under no condition: loads that only sometimes happen would
// make every wait one for all loads in flight.
template <class Operand, class Source, int DEPTH, int NW, class Open, class Load, class Multiply, class Begin, class Finish>
__device__ __forceinline__ void stream(int items, Open open, Load load, Multiply multiply, Begin begin, Finish finish) {
  if (items <= 0) return;
  Operand o[DEPTH];
  int block[DEPTH];                // the operands' blocks; -1: none
#pragma unroll
  for (int k = 0; k < DEPTH; ++k) block[k] = -1;
  Source src{};
  int ahead = -1, turns = 0;       // the item that loads are at, and its turns of DEPTH blocks left
#pragma nounroll
  while (true) {
    const bool enter = turns == 0;
    if (enter) {
      turns = 1;
      if (++ahead < items) {
        src = open(ahead);
        turns = max(1, (src.end - src.first + DEPTH * NW - 1) / (DEPTH * NW));
      }
    }
#pragma unroll
    for (int k = 0; k < DEPTH; ++k) {
      if (block[k] >= 0) multiply(block[k], o[k]);
      const int b = min(src.first, src.end - 1);   // past its end an item's last block is read again
      load(src, b, o[k]);
      block[k] = src.first < src.end ? b : -1;
      src.first += NW;
    }
    --turns;
    if (enter) {
      if (ahead > 0) finish(ahead - 1);
      if (ahead >= items) return;
      begin(ahead);
    }
  }
}

// A workgroup's share of the items (segment, row block), of kCus workgroups: a
// contiguous range.  Up to 32 segments share the workgroups out among
// themselves, since to ready a segment's activations costs as much as several
// items, and a range that runs on into the next segment does it twice (8
// experts of 11008 x 4096, 16 tokens each: 60 us, against 43); of more the
// shares would differ by more than that (100 segments: 2 or 3 workgroups each).
struct Share {
  unsigned first, n;               // items: number segment * n_rb + row block
};
__device__ inline Share share_of(unsigned segs, unsigned n_rb) {
  const unsigned wg = blockIdx.x;
  if (segs == 0) return {0, 0};
  if (segs > 32) {
    const unsigned all = segs * n_rb;
    auto upto = [&](unsigned b) { return all / kCus * b + all % kCus * b / kCus; };
    return {upto(wg), upto(wg + 1) - upto(wg)};
  }
  const unsigned sg = wg * segs / kCus;
  const unsigned first = (sg * kCus + segs - 1) / segs, n = ((sg + 1) * kCus + segs - 1) / segs - first;
  auto upto = [&](unsigned j) { return n_rb / n * j + n_rb % n * j / n; };
  return {sg * n_rb + upto(wg - first), upto(wg - first + 1) - upto(wg - first)};
}

// Eight of X's bf16 values of which the first is wanted at element `past`, of 0 .. 7.
__device__ inline u32x4 shifted_row(u32x4 v, int past) {
  if (past & 4) v[0] = v[2], v[1] = v[3];
  if (past & 2) v[0] = v[1], v[1] = v[2], v[2] = v[3];
  if (past & 1)
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = v[k] >> 16 | (k < 3 ? v[k + 1] << 16 : 0u);
  return v;
}

// The value of lane ^ 1 or ^ 2.
__device__ inline float quad1(float v) { return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xf, 0xf, true)); }
__device__ inline float quad2(float v) { return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xf, 0xf, true)); }
// The value of a lane of the other four of eight, where four hold the same.
__device__ inline float octet(float v) { return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xf, 0xf, true)); }

}  // namespace

#endif  // HINM_STREAM_H_
