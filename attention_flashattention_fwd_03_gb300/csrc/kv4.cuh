// kv4.cuh -- the 4-bit paged KV cache: format and quantiser, shared by every kernel
// that writes or reads it.
//
// Format.  32 consecutive channels of one (token, KV head) share a scale
//   s = amax / 7 rounded to 5 significant bits (ties to even), held as bf16
//   n = clamp(round(x / s), -7, 7), held as the code n + 8
// and stand for n s.  |n| takes 3 bits and s 5, so n s has at most 8 significant bits:
// every value the cache stands for is a bf16, which lets the prefill kernel hand exact
// operands to the tensor cores while the decode kernel keeps n and s apart, and both
// compute the same attention.  A group that holds a NaN or an infinity gets s = NaN and
// reads as NaN throughout; a group of zeros reads as zeros.
//
// A pool is [num_pool_blocks, Hkv, 18 D] bytes.  One (block, KV head) chunk holds
//   K codes  [16 tokens][D / 2]     K scales [16][D / 32] bf16
//   V codes  [16 tokens][D / 2]     V scales [16][D / 32] bf16
// contiguously (2304 bytes at D = 128, 1152 at D = 64, 28 % of the bf16 cache), so a
// block arrives with one untiled bulk copy.  Two codes share a byte, the even position
// low.  The order of the codes of a row is the order in which the decode kernel's
// matrix fragments take them straight from shared memory:
//   K: channel c at position ((c % 32) / 8 * (D / 32) + c / 32) * 8 + c % 8
//      -- the thread t = 0..3 of a row reads its D / 32 words (one a group) in one load
//   V: channel c at position ((c % 32) / 4 * (D / 32) + c / 32) * 4 + c % 4
//      -- the thread g = 0..7 of a dim reads 4 channels of every group in one load
#pragma once

#include <cstdint>

#include "paged.cuh"

namespace gbattn {

template <int D>
struct Kv4 {
  static constexpr int kGroup = 32;                      // channels that share a scale
  static constexpr int kGroups = D / kGroup;
  static constexpr int kCodeRow = D / 2;                 // bytes of a row's codes
  static constexpr int kScaleRow = kGroups * 2;          // bytes of a row's scales
  static constexpr int kOffKCodes = 0;
  static constexpr int kOffKScales = kPagedBlock * kCodeRow;
  static constexpr int kOffVCodes = kOffKScales + kPagedBlock * kScaleRow;
  static constexpr int kOffVScales = kOffVCodes + kPagedBlock * kCodeRow;
  static constexpr int kChunk = kOffVScales + kPagedBlock * kScaleRow;
  static_assert(kChunk == 18 * D, "the pool's last dimension");
};

// Scale of a group whose largest magnitude is amax (amax_bits = its bf16 bits without
// the sign; NaN and infinity compare above every finite value): fp32 bits whose low 16
// are zero, so the bf16 is the high half.
__device__ __forceinline__ uint32_t kv4_scale_bits(uint32_t amax_bits) {
  if (amax_bits >= 0x7f80u) return 0x7fc00000u;
  // a product with fp32(1 / 7) rounds to the same 5 bits as the quotient for each of the 128
  // significands of a bf16; subnormal quotients take the division
  const float a = __uint_as_float(amax_bits << 16);
  const uint32_t t = __float_as_uint(amax_bits >= 0x0400u ? a * (1.f / 7.f) : __fdiv_rn(a, 7.f));
  return (t + 0x3ffffu + ((t >> 19) & 1u)) & 0xfff80000u;  // 1 + 4 mantissa bits
}

// Codes of the eight channels of a lane for their group's scale (code 8, i.e. zero, where
// the scale is 0 or NaN), the first in the lowest nibble.
//
// n = round(x / s), ties to even, without a division: x has 8 significant bits and s 5,
// so a quotient that is not exactly k + 1/2 keeps a distance of at least 1/992 from it,
// while x (1 / s) is within 2^-21 of the quotient.  Adding 6144 rounds that product to a
// multiple of 2^-11, which puts exact ties back in place; adding 3 * 2^22 + 8 then rounds
// to an integer, whose low bits are the code.  (Checked against exact division for every
// pair of significands.)  |n| <= 7 holds by itself: s >= amax / 7 * 31 / 32.  Scales near
// the ends of the fp32 range, where 1 / s is not a normal number, take a division.
__device__ __forceinline__ uint32_t kv4_codes(const float2 (&x)[4], float s) {
  uint32_t w = 0;
  if (s > 1e-30f && s < 1e30f) {
    const float inv = __frcp_rn(s);
#pragma unroll
    for (int i = 3; i >= 0; --i) {
      float2 q = __ffma2_rn(x[i], make_float2(inv, inv), make_float2(6144.f, 6144.f));
      q = __fadd2_rn(q, make_float2(-6144.f, -6144.f));
      q = __fadd2_rn(q, make_float2(12582920.f, 12582920.f));
      w = 16 * w + __float_as_uint(q.y);
      w = 16 * w + __float_as_uint(q.x);
    }
    return w - 0x3f400000u;  // the sum of 0x4b400000 16^i
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = (i & 1) ? x[i / 2].y : x[i / 2].x;
    const float n = s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(v, s)), -7.f), 7.f) : 0.f;
    w |= static_cast<uint32_t>(static_cast<int>(n) + 8) << (4 * i);
  }
  return w;
}

// Eight codes u of one word (low nibble first) times a scale pair (s, s; bf16 bits): the
// bf16 values (u - 8) s TIMES / 64 in channel order, TIMES = 1 or 64.  A code alone in 16
// bits is the subnormal bf16 u 2^-133; one fused multiply-add makes it (u - 8) / 64 and the
// products scale it, all exact.  (TIMES = 1: where s >= 2^-123; below that a value / 64 is a
// subnormal bf16 and rounded to a multiple of 2^-133, so the value is off by 2^-128 at most.)  (The other way, 128 + u by an
// OR into the mantissa, then - 136, times s, delivers channels i and i + 4 in one register
// and takes four more permutes a word on the pipe that a softmax beside it needs: 784 us
// against 698 on the prefill of 16 x 512 tokens.)
template <int TIMES>
__device__ __forceinline__ uint4 kv4_values(uint32_t w, uint32_t s_bits) {
  static_assert(TIMES == 1 || TIMES == 64, "TIMES");
  const uint32_t big = 0x7f007f00u, off = 0xbe00be00u, times = 0x42804280u;  // 2^127, -2^-3, 64
  const uint32_t lo = w & 0x0f0f0f0fu, hi = (w >> 4) & 0x0f0f0f0fu;
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // bytes: low code, its sign (0), high code, its sign
    uint32_t u;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(u) : "r"(lo), "r"(hi), "r"(0xc480 + 0x1111 * i));
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(u) : "r"(u), "r"(big), "r"(off));
    if (TIMES == 64) asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(u) : "r"(u), "r"(times));
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(v[i]) : "r"(u), "r"(s_bits));
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

}  // namespace gbattn
