// attn_tile.cuh -- what the softmax warps of the tile kernels share: a score row of 128 keys
// a thread, read from and its probabilities written to tensor memory.
#pragma once

#include <cuda_runtime.h>

#include "ptx.cuh"

// With GBATTN_EXP2_POLY_PAIRS = n > 0, one key pair in every n of an unmasked
// tile has its probabilities computed on the FMA pipe (exp2_fma2) instead of
// the special-function unit.  Measured on GB300 the kernel is limited by issue
// slots and latency rather than by the special-function unit, and every setting
// tried (n = 2, 3, 4) was slower than 0, so it is off by default.
#ifndef GBATTN_EXP2_POLY_PAIRS
#define GBATTN_EXP2_POLY_PAIRS 0
#endif

namespace gbattn {

// (see reg_fence16)
__device__ __forceinline__ void reg_fence32(uint32_t (&r)[32]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31]));
}

// Keeps the compiler from using TMEM-load results before tcgen05.wait::ld.
__device__ __forceinline__ void reg_fence16(uint32_t (&r)[16]) {
  asm volatile(""
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// Largest score of a row.
__device__ __forceinline__ float row_max(const float (&s)[128]) {
  float mx0 = fmax3(s[0], s[1], s[2]), mx1 = fmax3(s[3], s[4], s[5]);
  float mx2 = fmax3(s[6], s[7], s[8]), mx3 = fmax3(s[9], s[10], s[11]);
#pragma unroll
  for (int c = 12; c < 124; c += 8) {
    mx0 = fmax3(mx0, s[c], s[c + 1]);
    mx1 = fmax3(mx1, s[c + 2], s[c + 3]);
    mx2 = fmax3(mx2, s[c + 4], s[c + 5]);
    mx3 = fmax3(mx3, s[c + 6], s[c + 7]);
  }
  mx0 = fmax3(mx0, s[124], s[125]);
  mx1 = fmax3(mx1, s[126], s[127]);
  return fmax3(fmaxf(mx0, mx1), mx2, mx3);
}

// Probabilities of one row: p = 2^(c s - c m) for the 128 keys of the tile,
// summed in fp32 and written to TMEM (at p_addr) as bf16 pairs over the upper
// half of S.  Keys are handled in pairs with the packed fp32x2 instructions.
// With POLY (tiles without masked keys) one pair in GBATTN_EXP2_POLY_PAIRS uses
// the FMA-pipe exp2; masked keys (s = -inf) always go through ex2, which gives
// exactly 0 for them.
template <bool POLY>
__device__ __forceinline__ void write_p(const float (&s)[128], float sl2, float ms,
                                        uint32_t p_addr, float2 (&sum)[2]) {
  const float2 k2 = make_float2(sl2, sl2), m2 = make_float2(-ms, -ms);
  constexpr int kEvery = GBATTN_EXP2_POLY_PAIRS > 0 ? GBATTN_EXP2_POLY_PAIRS : 1;
#pragma unroll
  for (int ch = 0; ch < 8; ++ch) {  // 16 keys -> 8 packed columns per chunk
    uint32_t pk[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c0 = 16 * ch + 2 * e;
      const float2 x = __ffma2_rn(make_float2(s[c0], s[c0 + 1]), k2, m2);
      float2 pr;
      if (POLY && GBATTN_EXP2_POLY_PAIRS > 0 && (c0 / 2) % kEvery == kEvery - 1)
        pr = exp2_fma2(x);
      else
        pr = make_float2(ex2(x.x), ex2(x.y));
      sum[e & 1] = __fadd2_rn(sum[e & 1], pr);
      pk[e] = pack_bf16x2(pr.x, pr.y);
    }
    tmem_st8(p_addr + 8 * ch, pk);
  }
}

}  // namespace gbattn
