// decode_split.cuh -- how a paged decode shares the batch's cache between warps, for the
// bf16 and the 4-bit kernels.
//
// All (request, KV head, 16-token block) triples form one sequence, request-major; it
// is cut into W equal contiguous ranges, one per consumer warp.  A range may cross from
// one (request, KV head) segment into the next; a warp ends a "piece" there.  The ranges
// depend only on the sequence lengths of the batch.
#pragma once

#include "internal.h"
#include "paged.cuh"

namespace gbattn {

// Blocks per KV head of a request of L tokens; 0 for a length outside its bounds
// (the merge kernel reports that request).
__device__ __forceinline__ int blocks_of(const DecodeParams& p, int L) {
  return (L < 0 || L > p.max_seq_len || L > p.max_blocks * kPagedBlock)
             ? 0
             : (L + kPagedBlock - 1) / kPagedBlock;
}

// The warp range holding block b of the global order: ranges are
// [floor(k NB / W), floor((k + 1) NB / W)), so this is the largest k whose range
// starts at or before b.
__device__ __forceinline__ int range_of(long long b, long long NB, int W) {
  return static_cast<int>(((b + 1) * W - 1) / NB);
}

// A position in the global (request, KV head, block) order.
struct Cursor {
  long long first;  // global index of block 0 of segment (r, h)
  int r, h, b, nb;
};

// Moves c forward by k blocks.  The caller guarantees the target lies inside the
// order; should the lengths say otherwise, r stops at S and the caller's checks
// see it.
__device__ __forceinline__ void advance(Cursor& c, int k, const DecodeParams& p) {
  c.b += k;
  while (c.b >= c.nb && c.r < p.S) {
    c.b -= c.nb;
    c.first += c.nb;
    if (++c.h == p.Hkv) {
      c.h = 0;
      c.nb = 0;
      while (c.nb == 0 && ++c.r < p.S) c.nb = blocks_of(p, p.seq_lens[c.r]);
    }
  }
}

// --------------------------------------------------------------------------
// warp-level matrix products (m16n8k16, bf16 inputs, fp32 accumulators)
// --------------------------------------------------------------------------
// D = A * B + D
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

}  // namespace gbattn
