// norm_rope.cuh -- RMS norm and position rotation of one head's row, shared by the
// forward and cache-append kernels so they agree bit for bit, and the backward kernel.
//
//   xh = x * rsqrt(mean(x^2) + eps)      y = R(pos) (xh * w)
// over the D channels of one (token, head); without a weight y = R(pos) x.  R turns the
// first `rot` channels as rot / 2 planes: plane i pairs channels (i, i + rot / 2), or
// (2 i, 2 i + 1) when interleaved, and
//   y_a = x_a cos_i - x_b sin_i      y_b = x_b cos_i + x_a sin_i
// with cos_i, sin_i from row pos of the table [max_pos, rot] (cos first, then sin).
// The table's values may carry any factor (scaled rotations); its transpose is what the
// backward pass applies.
//
// D / 8 lanes share a row, 8 channels a lane in two runs of 4, placed so that both
// channels of a plane sit in one lane: lane l < rot / 8 holds channels 4 l.. and
// rot / 2 + 4 l.. (8 l.. and 8 l + 4.. when interleaved), the lanes past the rotated
// part 8 l.. and 8 l + 4...  Either way a rotating lane uses planes 4 l .. 4 l + 3, and
// the rotation needs no exchange between lanes.  rot is a multiple of 8 for this.
//
// All arithmetic is fp32; a row is rounded to bf16 once, after the rotation.  Up to there
// the forward takes the formula's operations one by one, x r, times w, two products and
// their sum, each rounded, as a program that evaluates it tensor by tensor does: a fused
// product would differ in the last bit of one value in some ten thousand, which the 4-bit
// cache can turn into a whole step.  (Costs 0.4 of 66 us on a 16k prompt, 1 of 50 on an
// append to the 4-bit cache and its gather.)  The exception is the sum of squares behind r
// where a row turns in part or interleaved: fused products, in the order of the lanes.  It is
// as exact, but not the same bits: a row may differ in its last bit between such a rotation
// and a full one of halves (row_squares).
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace gbattn {

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

constexpr uint32_t kBf16NanPair = 0x7fc07fc0u;

// Channels of one lane: runs of 4 starting at c0 and c1, and whether it rotates.
struct LaneChannels {
  int c0, c1;
  bool rotates;
};

__device__ __forceinline__ LaneChannels lane_channels(int l, int rot, int interleaved) {
  LaneChannels c;
  c.rotates = 8 * l < rot;
  const bool split = c.rotates && !interleaved;
  c.c0 = split ? 4 * l : 8 * l;
  c.c1 = split ? 4 * l + rot / 2 : 8 * l + 4;
  return c;
}

// A lane's eight channels as fp32 pairs, for the packed fp32x2 instructions: the first
// run of 4 in v[0], v[1], the second in v[2], v[3].
struct Lane8 {
  float2 v[4];
};

__device__ __forceinline__ float2 widen2(uint32_t w) { return make_float2(bf16_lo(w), bf16_hi(w)); }

__device__ __forceinline__ Lane8 widen8(uint2 a, uint2 b) {
  return Lane8{{widen2(a.x), widen2(a.y), widen2(b.x), widen2(b.y)}};
}

__device__ __forceinline__ void round8(const Lane8& x, uint2& a, uint2& b) {
  a = make_uint2(pack_bf16x2(x.v[0].x, x.v[0].y), pack_bf16x2(x.v[1].x, x.v[1].y));
  b = make_uint2(pack_bf16x2(x.v[2].x, x.v[2].y), pack_bf16x2(x.v[3].x, x.v[3].y));
}

__device__ __forceinline__ Lane8 mul8(const Lane8& x, const Lane8& y) {
  Lane8 z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.v[i] = __fmul2_rn(x.v[i], y.v[i]);
  return z;
}

__device__ __forceinline__ Lane8 scale8(const Lane8& x, float f) {
  Lane8 z;
#pragma unroll
  for (int i = 0; i < 4; ++i) z.v[i] = __fmul2_rn(x.v[i], make_float2(f, f));
  return z;
}

// This lane's part of the dot product of two rows.
__device__ __forceinline__ float dot8(const Lane8& x, const Lane8& y) {
  float2 s = __fmul2_rn(x.v[0], y.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = __ffma2_rn(x.v[i], y.v[i], s);
  return s.x + s.y;
}

// Sum over the LANES lanes that share a row; every lane gets the same bits.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// cos and sin of a lane's four planes (BACK: of the transposed rotation).
struct Planes {
  float2 c[2], s[2];
};

// x y + z u with both products and the sum rounded.  The sum is a multiply-add by a one that
// the compiler does not know: it joins a packed product and a packed sum to one operation.
__device__ __forceinline__ float2 rounded_sum2(float2 x, float2 y, float2 z, float2 u, float one) {
  return __ffma2_rn(__fmul2_rn(z, u), make_float2(one, one), __fmul2_rn(x, y));
}

// Turns the lane's four planes, every operation rounded by itself.
__device__ __forceinline__ void rotate8_stepwise(Lane8& x, const Planes& p, int interleaved,
                                                 float one) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = x.v[i], b = x.v[2 + i];
      const float2 ns = make_float2(-p.s[i].x, -p.s[i].y);
      x.v[i] = rounded_sum2(a, p.c[i], b, ns, one);
      x.v[2 + i] = rounded_sum2(b, p.c[i], a, p.s[i], one);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = (i & 1) ? p.c[i / 2].y : p.c[i / 2].x, s = (i & 1) ? p.s[i / 2].y : p.s[i / 2].x;
      const float a = x.v[i].x, b = x.v[i].y;
      x.v[i] = make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)),
                           __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
    }
  }
}

// Sum of the squares of a row.  FULL (every channel rotates, planes of halves): 32 columns
// c, c + 32, .. are added first, then neighbouring columns in pairs, the order in which a
// reduction over a row of 128 or 64 values by a warp goes, for the reason given above.  Else
// a lane's eight are added with fused products, then the lanes.
template <int D, bool FULL>
__device__ __forceinline__ float row_squares(const Lane8& x, int l) {
  if constexpr (!FULL) {
    return row_sum<D / 8>(dot8(x, x));
  } else {
    const Lane8 q = mul8(x, x);  // exact: x is bf16
    float s;
    if constexpr (D == 64) {
      const float2 z0 = __fadd2_rn(q.v[0], q.v[2]), z1 = __fadd2_rn(q.v[1], q.v[3]);
      s = (z0.x + z0.y) + (z1.x + z1.y);
    } else {
      // lanes l and l + 8 hold quarters 0, 2 and 1, 3 of the same four columns: each adds two
      const bool up = l & 8;
      const float2 give0 = up ? q.v[0] : q.v[1], give1 = up ? q.v[2] : q.v[3];
      const float2 own0 = up ? q.v[1] : q.v[0], own1 = up ? q.v[3] : q.v[2];
      float2 got0, got1;
      got0.x = __shfl_xor_sync(0xffffffffu, give0.x, 8);
      got0.y = __shfl_xor_sync(0xffffffffu, give0.y, 8);
      got1.x = __shfl_xor_sync(0xffffffffu, give1.x, 8);
      got1.y = __shfl_xor_sync(0xffffffffu, give1.y, 8);
      const float2 z = __fadd2_rn(__fadd2_rn(__fadd2_rn(own0, got0), up ? got1 : own1), up ? own1 : got1);
      s = z.x + z.y;
      s += __shfl_xor_sync(0xffffffffu, s, 8);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
  }
}

// Turns the lane's four planes.
__device__ __forceinline__ void rotate8(Lane8& x, const Planes& p, int interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = x.v[i], b = x.v[2 + i];
      const float2 ns = make_float2(-p.s[i].x, -p.s[i].y);
      x.v[i] = __ffma2_rn(b, ns, __fmul2_rn(a, p.c[i]));
      x.v[2 + i] = __ffma2_rn(a, p.s[i], __fmul2_rn(b, p.c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float c = (i & 1) ? p.c[i / 2].y : p.c[i / 2].x, s = (i & 1) ? p.s[i / 2].y : p.s[i / 2].x;
      const float a = x.v[i].x, b = x.v[i].y;
      x.v[i] = make_float2(fmaf(b, -s, a * c), fmaf(a, s, b * c));
    }
  }
}

}  // namespace gbattn
