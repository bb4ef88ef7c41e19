// norm_rope.cuh -- RMS norm and position rotation of one head's row, shared by the
// forward, backward and cache-append kernels so they agree bit for bit.
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
// All arithmetic is fp32; a row is rounded to bf16 once, after the rotation.
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

// Eight packed bf16 of a lane (two runs of 4) -> fp32.
__device__ __forceinline__ void widen8(uint2 a, uint2 b, float (&x)[8]) {
  x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
  x[4] = bf16_lo(b.x), x[5] = bf16_hi(b.x), x[6] = bf16_lo(b.y), x[7] = bf16_hi(b.y);
}

__device__ __forceinline__ void round8(const float (&x)[8], uint2& a, uint2& b) {
  a = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
  b = make_uint2(pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// Sum over the LANES lanes that share a row; every lane gets the same bits.
template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// 1 / rms of a row from this lane's 8 channels.
template <int D>
__device__ __forceinline__ float row_rrms(const float (&x)[8], float eps) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = fmaf(x[i], x[i], s);
  return rsqrtf(row_sum<D / 8>(s) * (1.f / D) + eps);
}

// Turns the lane's four planes by cos / sin (BACK: by the transpose).
template <bool BACK>
__device__ __forceinline__ void rotate8(float (&x)[8], float4 co, float4 si, int interleaved) {
  const float c[4] = {co.x, co.y, co.z, co.w};
  const float s[4] = {si.x, si.y, si.z, si.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float sn = BACK ? -s[i] : s[i];
    if (interleaved) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * c[i] - b * sn;
      x[2 * i + 1] = b * c[i] + a * sn;
    } else {
      const float a = x[i], b = x[4 + i];
      x[i] = a * c[i] - b * sn;
      x[4 + i] = b * c[i] + a * sn;
    }
  }
}

}  // namespace gbattn
