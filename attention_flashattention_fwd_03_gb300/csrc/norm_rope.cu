// norm_rope.cu -- from a model's QKV projection to what the attention kernels read:
// per-head RMS norm, position rotation and relayout in one pass, with its gradients, and
// the same pass writing K and V straight into the paged caches (bf16 or 4 bits).
// The mathematics and the lane layout are in norm_rope.cuh, the 4-bit format in kv4.cuh.
//
// Forward and appends: memory-bound, each value read and written once.  A warp takes a
// run of the rows (q, k and v heads) of one token, 32 / (D / 8) rows a pass, so its table
// row and weights are read once and every row moves as whole 128- or 256-byte segments;
// the loads of four passes are in flight together.  D 128: a 16k prompt of 32/8 heads (411
// MB) 66 us, 91 % of the copy rate; 16 x 512 tokens appended to the bf16 cache (202 MB) 36 us,
// 83 %; to the 4-bit cache (187 MB) 40 us, 69 %: a quarter more instructions (64 % of the issue
// slots), and K rows pass through shared memory between two warp barriers a row set, which
// puts the passes in flight back in line.  Neither HBM nor the issue slots are full.
#include <cuda_runtime.h>

#include <type_traits>

#include "kv4.cuh"
#include "norm_rope.cuh"
#include "norm_rope.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

// One warp a CTA: a token's rows leave an SM as they end, without waiting for others.
// (16k prompt, four passes unrolled: 1 warp 66.1 us, 2 68.4, 4 68.6, 8 69.6, each held to
// 64 registers; two passes unrolled 77.5, three 75.0, six 74.3, eight 91.8.)  CTAs an SM
// (registers), 16k prompt / bf16 append / 4-bit append and gather of 16 x 512 tokens: 32 (64)
// 66.4 / 36.0 / 49.9 us, 28 (72) 66.1 / 36.3 / 48.7, 24 (80) 67.9 / 36.1 / 53.7, 20 78.9 / 41.8 / 54.6.
constexpr int kWarps = 1;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 28;

__device__ __forceinline__ uint2 ld8(const uint16_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ void st8(uint16_t* p, uint2 v) { *reinterpret_cast<uint2*>(p) = v; }

// Table entries of the lane's four planes (1 and 0 for a lane that does not rotate);
// BACK: of the transposed rotation.
template <bool BACK>
__device__ __forceinline__ Planes load_planes(const RopeParams& r, int pos, int l, bool rotates) {
  float4 co = make_float4(1.f, 1.f, 1.f, 1.f), si = make_float4(0.f, 0.f, 0.f, 0.f);
  if (rotates) {
    const float* row = r.cos_sin + static_cast<size_t>(pos) * r.rot;
    co = *reinterpret_cast<const float4*>(row + 4 * l);
    si = *reinterpret_cast<const float4*>(row + r.rot / 2 + 4 * l);
  }
  const float f = BACK ? -1.f : 1.f;
  return Planes{{make_float2(co.x, co.y), make_float2(co.z, co.w)},
                {make_float2(f * si.x, f * si.y), make_float2(f * si.z, f * si.w)}};
}

// Quantises one row of D bf16 (the lane's 8 channels from 8 l on, packed) into a chunk
// of the 4-bit pool, as a K or a V row of token slot `slot`.  All lanes take part;
// `write` is the same over a row.
template <int D, bool IS_V>
__device__ __forceinline__ void quantise_row(uint4 w, uint8_t* chunk, int slot, int l, bool write) {
  using F = Kv4<D>;
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  // bf16 magnitudes order like their bits, NaN and infinity on top
  uint32_t pair = __vmaxu2(__vmaxu2(in[0] & 0x7fff7fffu, in[1] & 0x7fff7fffu),
                           __vmaxu2(in[2] & 0x7fff7fffu, in[3] & 0x7fff7fffu));
  pair = __vmaxu2(pair, __shfl_xor_sync(0xffffffffu, pair, 1));
  pair = __vmaxu2(pair, __shfl_xor_sync(0xffffffffu, pair, 2));
  const uint32_t sbits = kv4_scale_bits(max(pair & 0xffffu, pair >> 16));
  float2 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = widen2(in[i]);
  const uint32_t codes = kv4_codes(x, __uint_as_float(sbits));
  if (!write) return;
  const int group = l >> 2, part = l & 3;  // channels 8 l .. 8 l + 7 of group l / 4
  uint8_t* row = chunk + (IS_V ? F::kOffVCodes : F::kOffKCodes) + slot * F::kCodeRow;
  if constexpr (IS_V) {
    uint16_t* h = reinterpret_cast<uint16_t*>(row);
    h[(2 * part) * F::kGroups + group] = static_cast<uint16_t>(codes & 0xffffu);
    h[(2 * part + 1) * F::kGroups + group] = static_cast<uint16_t>(codes >> 16);
  } else {
    reinterpret_cast<uint32_t*>(row)[part * F::kGroups + group] = codes;
  }
  if (part == 0) {
    uint8_t* sc = chunk + (IS_V ? F::kOffVScales : F::kOffKScales) + slot * F::kScaleRow;
    reinterpret_cast<uint16_t*>(sc)[group] = static_cast<uint16_t>(sbits >> 16);
  }
}

constexpr int kUnroll = 4;  // passes whose loads are in flight together

// What the rows of one token share.
struct TokenCtx {
  LaneChannels ch;
  Planes planes;
  int l, sub;       // lane within its row, row within the pass
  int interleaved;
  float eps, one;   // (one: for rounded_sum2)
  bool live;        // false: q and k rows are NaN
  bool write_kv;    // paged: K and V reach the cache
  int slot;
};

// Query or key rows h0 .. h1 - 1: x[h * sh] -> y[h * oh] (QUANT: the 4-bit chunk at
// y4 + h * kChunk, through the warp's rows of shared memory, which bring the lane's two
// runs of channels into order).  Lanes whose row lies past h1 take part with zeros.
template <int D, bool QUANT, bool FULL>
__device__ __forceinline__ void norm_rope_rows(const TokenCtx& t, const uint16_t* x, long long sh,
                                               const uint16_t* w, int h0, int h1, uint16_t* y,
                                               long long oh, uint8_t* y4, uint16_t* stage,
                                               bool write) {
  constexpr int LANES = D / 8;
  constexpr int ROWS = 32 / LANES;
  Lane8 wf{};
  if (w) wf = widen8(ld8(w + t.ch.c0), ld8(w + t.ch.c1));
  for (int r0 = h0; r0 < h1; r0 += ROWS * kUnroll) {
    uint2 a[kUnroll], c[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = r0 + u * ROWS + t.sub;
      a[u] = c[u] = make_uint2(0, 0);
      if (h < h1) {
        a[u] = ld8(x + h * sh + t.ch.c0);
        c[u] = ld8(x + h * sh + t.ch.c1);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * ROWS >= h1) break;
      const int h = r0 + u * ROWS + t.sub;
      Lane8 v = widen8(a[u], c[u]);
      if (w) {
        const float r = rsqrtf(row_squares<D, FULL>(v, t.l) * (1.f / D) + t.eps);
        v = mul8(scale8(v, r), wf);
      }
      if (FULL || t.ch.rotates) rotate8_stepwise(v, t.planes, FULL ? 0 : t.interleaved, t.one);
      round8(v, a[u], c[u]);
      if (!t.live) a[u] = c[u] = make_uint2(kBf16NanPair, kBf16NanPair);
      if constexpr (QUANT) {
        uint16_t* mine = stage + t.sub * D;
        __syncwarp();
        st8(mine + t.ch.c0, a[u]);
        st8(mine + t.ch.c1, c[u]);
        __syncwarp();
        quantise_row<D, false>(*reinterpret_cast<const uint4*>(mine + 8 * t.l),
                               y4 + h * static_cast<long long>(Kv4<D>::kChunk), t.slot, t.l,
                               write && h < h1);
      } else if (write && h < h1) {
        st8(y + h * oh + t.ch.c0, a[u]);
        st8(y + h * oh + t.ch.c1, c[u]);
      }
    }
  }
}

// Value rows h0 .. h1 - 1, taken in channel order.
template <int D, bool QUANT>
__device__ __forceinline__ void value_rows(const TokenCtx& t, const uint16_t* x, long long sh,
                                           int h0, int h1, uint16_t* y, long long oh, uint8_t* y4,
                                           bool write) {
  constexpr int LANES = D / 8;
  constexpr int ROWS = 32 / LANES;
  for (int r0 = h0; r0 < h1; r0 += ROWS * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = r0 + u * ROWS + t.sub;
      v[u] = make_uint4(0, 0, 0, 0);
      if (h < h1) v[u] = *reinterpret_cast<const uint4*>(x + h * sh + 8 * t.l);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * ROWS >= h1) break;
      const int h = r0 + u * ROWS + t.sub;
      if constexpr (QUANT) {
        quantise_row<D, true>(v[u], y4 + h * static_cast<long long>(Kv4<D>::kChunk), t.slot, t.l,
                              write && h < h1);
      } else if (write && h < h1) {
        *reinterpret_cast<uint4*>(y + h * oh + 8 * t.l) = v[u];
      }
    }
  }
}

template <int D, RowSink SINK, bool FULL>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LANES = D / 8;       // lanes of one row
  constexpr int ROWS = 32 / LANES;   // rows of one pass
  constexpr bool PAGED = SINK != RowSink::kContiguous;
  constexpr bool QUANT = SINK == RowSink::kPaged4;
  __shared__ __align__(16) uint16_t stage[QUANT ? kWarps * ROWS * D : 8];
  // a kernel launched next as a programmatic dependent (a decode behind an append) may start
  // its set-up now; it waits for this grid's writes before it reads anything, as this one
  // does for the grid before.  (Not the forward: followed by itself on odd sizes it takes
  // 5.5 us so, 4.1 without.)
  if (PAGED) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long wid = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long tok = wid / p.chunks;
  const int chunk = static_cast<int>(wid - tok * p.chunks);
  if (tok >= static_cast<long long>(p.B) * p.T) return;
  const int b = static_cast<int>(tok / p.T), ti = static_cast<int>(tok - static_cast<long long>(b) * p.T);
  TokenCtx t;
  t.l = lane % LANES;
  t.sub = lane / LANES;
  t.interleaved = p.rope.interleaved;
  t.eps = p.rope.eps;
  t.one = p.one;
  t.ch = lane_channels(t.l, p.rope.rot, p.rope.interleaved);
  t.live = t.write_kv = true;
  t.slot = 0;

  // ---- where this token goes, and its rotation ----
  int pos = ti;
  long long block = 0;    // paged: physical block
  const bool first = chunk == 0 && lane == 0;
  if constexpr (PAGED) {
    const int L = p.seq_lens[b];
    if (L < 0 || L > p.max_blocks * kPagedBlock - p.T) {
      if (first && ti == 0) {
        raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
        if (p.new_seq_lens) p.new_seq_lens[b] = L;
      }
      t.live = t.write_kv = false;
    } else {
      if (first && ti == 0 && p.new_seq_lens) p.new_seq_lens[b] = L + p.T;
      pos = L + ti;
      t.slot = pos % kPagedBlock;
      block = p.block_table[static_cast<size_t>(b) * p.max_blocks + pos / kPagedBlock];
      if (block < 0 || block >= p.num_pool_blocks) {
        if (first) raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
        t.write_kv = false;
        block = 0;
      }
    }
  }
  if (p.rope.rot > 0 && t.live) {
    if (p.rope.positions) pos = p.rope.positions[tok];
    if (pos < 0 || pos >= p.rope.max_pos) {
      if (first) raise_flag(p.flags, DEVFLAG_BAD_POSITION);
      t.live = false;
      if (PAGED) t.write_kv = false;
    }
  }
  t.planes = load_planes<false>(p.rope, pos, t.l, t.ch.rotates && t.live);

  // ---- this warp's share of the token's query, key and value rows ----
  const int rows = p.nq + p.nk + p.nv;
  const int c0 = chunk * p.rows_per_warp, c1 = min(rows, c0 + p.rows_per_warp);
  auto in = [&](const Heads& x) { return x.p + b * x.sb + ti * x.st; };
  auto out = [&](uint16_t* y, int heads) {
    return y + (static_cast<long long>(b) * heads * p.T + ti) * D;
  };
  const long long oh = static_cast<long long>(p.T) * D;
  if (c0 < p.nq)
    norm_rope_rows<D, false, FULL>(t, in(p.q), p.q.sh, p.rope.q_weight, c0, min(c1, p.nq),
                             out(p.q_out, p.nq), oh, nullptr, nullptr, true);
  const int k0 = max(c0 - p.nq, 0), k1 = min(c1 - p.nq, p.nk);
  const int v0 = max(c0 - p.nq - p.nk, 0), v1 = c1 - p.nq - p.nk;
  if constexpr (!PAGED) {
    if (k0 < k1)
      norm_rope_rows<D, false, FULL>(t, in(p.k), p.k.sh, p.rope.k_weight, k0, k1, out(p.k_out, p.nk), oh,
                               nullptr, nullptr, true);
    if (v0 < v1) value_rows<D, false>(t, in(p.v), p.v.sh, v0, v1, out(p.v_out, p.nv), oh, nullptr, true);
  } else if constexpr (!QUANT) {
    const long long at = (block * p.nk * kPagedBlock + t.slot) * D;  // pool row of head 0
    constexpr long long ph = kPagedBlock * D;
    if (k0 < k1)
      norm_rope_rows<D, false, FULL>(t, in(p.k), p.k.sh, p.rope.k_weight, k0, k1, p.k_pool + at, ph,
                               nullptr, nullptr, t.write_kv);
    if (v0 < v1)
      value_rows<D, false>(t, in(p.v), p.v.sh, v0, v1, p.v_pool + at, ph, nullptr, t.write_kv);
  } else {
    uint8_t* chunk4 = p.kv4_pool + block * p.nk * Kv4<D>::kChunk;
    if (k0 < k1)
      norm_rope_rows<D, true, FULL>(t, in(p.k), p.k.sh, p.rope.k_weight, k0, k1, nullptr, 0, chunk4,
                              stage + (threadIdx.x >> 5) * ROWS * D, t.write_kv);
    if (v0 < v1)
      value_rows<D, true>(t, in(p.v), p.v.sh, v0, v1, nullptr, 0, chunk4, t.write_kv);
  }
}

}  // namespace

// Launches as a programmatic dependent: the grid may be set up while the one before ends.
// (Every kernel here waits for that one before it reads or writes global memory.)  Calls in a
// row, us each, plainly launched / so: 16k prompt 68.1 / 66.1, backward 48.8 / 46.4, bf16
// append of 16 x 512 38.9 / 36.1, 4-bit append and gather 53.3 / 48.7, of 64 tokens 10.3 / 7.8.
template <typename K, typename... Args>
static cudaError_t launch_dependent(K* kernel, dim3 grid, dim3 block, size_t smem,
                                    cudaStream_t stream, const Args&... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_norm_rope(NormRopeParams p, int D, RowSink sink, int num_sms,
                             cudaStream_t stream) {
  const int rows = p.nq + p.nk + p.nv;
  const long long tokens = static_cast<long long>(p.B) * p.T;
  if (tokens <= 0 || rows <= 0) return cudaSuccess;
  // A warp takes whole tokens where there are enough of them to fill the SMs (the table
  // row and the weights are then read once), else four passes of a token, or two where
  // there are so few tokens that only the depth of the work counts.
  const int pass = 256 / D;
  p.rows_per_warp = tokens >= 32ll * num_sms ? rows : (tokens >= 4ll * num_sms ? 4 : 2) * pass;
  p.chunks = (rows + p.rows_per_warp - 1) / p.rows_per_warp;
  p.one = 1.f;
  const long long grid = (tokens * p.chunks + kWarps - 1) / kWarps;  // (its bound: too_many_rows)
  const dim3 g(static_cast<unsigned>(grid));
  auto run = [&](auto d, auto f) {
    constexpr int DD = decltype(d)::value;
    constexpr bool FULL = decltype(f)::value;
    auto* kernel = sink == RowSink::kContiguous
                       ? norm_rope_kernel<DD, RowSink::kContiguous, FULL>
                       : (sink == RowSink::kPaged ? norm_rope_kernel<DD, RowSink::kPaged, FULL>
                                                  : norm_rope_kernel<DD, RowSink::kPaged4, FULL>);
    return launch_dependent(kernel, g, dim3(kThreads), 0, stream, p);
  };
  auto sized = [&](auto f) {
    return D == 64 ? run(std::integral_constant<int, 64>{}, f)
                   : run(std::integral_constant<int, 128>{}, f);
  };
  return p.rope.rot == D && !p.rope.interleaved ? sized(std::true_type{}) : sized(std::false_type{});
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// With dy = R^T g (g the gradient of the rotated row), xh = x r and u = dy * w:
//   dx = r (u - xh mean(u xh))      dw = sum over tokens and heads of dy xh
// (no weight: dx = dy).  A warp takes one operand of one token at a time, so that the warps
// end together; the lane's eight channels are the same in every row, so the weight
// gradients stay in registers until the CTA has seen all of its tokens.  They are then
// summed over the CTA in shared memory and written as one partial per CTA; a second kernel
// adds the partials.  No atomics: the order of every sum depends on the sizes alone.
//
// Memory-bound (x and g read, dx written).  A warp streams its units pass by pass, a pass
// being 2 KB of g, 2 KB of x and the token's row of the table, through its own ring of
// stages in shared memory: the copies of the next passes are in flight while one is
// computed, which registers alone did not allow (57 us so).  4 x 2048 tokens of 16/16
// heads, D 128: 45.7 us for 269 MB, 87 % of the copy rate, about 2 of them the sum over the
// partials (read one after the other they took one more).  Two stages of four row sets 46.3 us, three 48.6; six stages of two sets 81,
// two of six 59, both with a pass's set-up costing more than its rows.
namespace {

constexpr int kBwdWarps = 8;
constexpr int kBwdThreads = kBwdWarps * 32;
constexpr int kBwdCtasPerSm = 2;
constexpr int kBwdMaxGrid = 304;  // two CTAs on each of 152 SMs
constexpr int kBwdUnroll = 4;  // row sets of a pass
constexpr int kBwdStages = 2;

template <int D>
struct BwdShape {
  static constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a set
  static constexpr int kHalf = kBwdUnroll * 512;             // bytes of a pass of g or of x
  static constexpr int kStage = 2 * kHalf + 4 * D;           // and a row of the table
  static constexpr int kSmem = kBwdWarps * kBwdStages * kStage;
  static_assert(kSmem >= kBwdWarps * kRows * 2 * D * 4, "the ring also holds the warps' sums");
};

// A row set of queries or keys: dx from the gradient and, with a weight, the input (both in
// shared memory); adds this lane's terms of the weight gradient to dw.
template <int D, bool INTERLEAVED, bool NORM>
__device__ __forceinline__ void norm_rope_bwd_set(const TokenCtx& t, const uint16_t* g,
                                                  const uint16_t* x, const uint2 (&w)[2],
                                                  uint16_t* dx, bool write, Lane8& dw) {
  constexpr int LANES = D / 8;
  Lane8 v = widen8(ld8(g + t.ch.c0), ld8(g + t.ch.c1));
  if (t.ch.rotates) rotate8(v, t.planes, INTERLEAVED);
  if constexpr (NORM) {
    const Lane8 x8 = widen8(ld8(x + t.ch.c0), ld8(x + t.ch.c1));
    const Lane8 vw = mul8(v, widen8(w[0], w[1]));
    // both sums of the row at once: x^2 and (dy w) x
    const float ss = row_sum<LANES>(dot8(x8, x8)), dot = row_sum<LANES>(dot8(vw, x8));
    const float r = rsqrtf(ss * (1.f / D) + t.eps);
    const float m = -dot * r * (1.f / D);
    const Lane8 xh = scale8(x8, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dw.v[i] = __ffma2_rn(v.v[i], xh.v[i], dw.v[i]);  // 0 for a row past the end: its g is 0
      v.v[i] = __ffma2_rn(xh.v[i], make_float2(m, m), vw.v[i]);
    }
    v = scale8(v, r);
  }
  uint2 a, c;
  round8(v, a, c);
  if (!t.live) a = c = make_uint2(kBf16NanPair, kBf16NanPair);
  if (write) {
    st8(dx, a);
    st8(dx + (t.ch.c1 - t.ch.c0), c);
  }
}

template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kBwdThreads, kBwdCtasPerSm)
    norm_rope_bwd_kernel(const NormRopeBwdParams p) {
  using C = BwdShape<D>;
  constexpr int LANES = C::kLanes, ROWS = C::kRows, PASS = kBwdUnroll * ROWS;
  extern __shared__ __align__(16) uint8_t smem[];
  // the sum over the partials may be scheduled now; it waits for this grid's results, as this
  // one does for those of the grid before
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * kBwdStages * C::kStage;
  const uint32_t ring_addr = smem_u32(ring) + lane * 16;
  TokenCtx t;
  t.l = lane % LANES;
  t.sub = lane / LANES;
  t.interleaved = INTERLEAVED;
  t.eps = p.rope.eps;
  t.ch = lane_channels(t.l, p.rope.rot, INTERLEAVED);
  t.live = true;
  uint2 wq[2] = {}, wk[2] = {};
  if (p.rope.q_weight) wq[0] = ld8(p.rope.q_weight + t.ch.c0), wq[1] = ld8(p.rope.q_weight + t.ch.c1);
  if (p.rope.k_weight) wk[0] = ld8(p.rope.k_weight + t.ch.c0), wk[1] = ld8(p.rope.k_weight + t.ch.c1);
  Lane8 dwq{}, dwk{};

  // Unit: operand op (0 q, 1 k, 2 v) of token ti of batch entry b; a warp takes every
  // gridDim.x * kBwdWarps-th unit.
  struct Unit {
    int b, ti, op;
  };
  const unsigned stride = gridDim.x * kBwdWarps, T = p.T;
  const int step_op = stride % 3, step_t = stride / 3 % T, step_b = stride / 3 / T;
  auto heads_of = [&](int op) { return op == 0 ? p.nq : (op == 1 ? p.nk : p.nv); };
  auto advance = [&](Unit& u) {  // to the warp's next unit that has rows
    do {
      u.op += step_op;
      u.ti += step_t + (u.op >= 3 ? 1 : 0);  // at most T - 1 + 1 more
      u.op -= u.op >= 3 ? 3 : 0;
      u.b += step_b;
      if (u.ti >= p.T) u.ti -= p.T, ++u.b;
    } while (u.b < p.B && heads_of(u.op) == 0);
  };
  const unsigned first = blockIdx.x * kBwdWarps + warp;
  Unit at{static_cast<int>(first / 3 / T), static_cast<int>(first / 3 % T), static_cast<int>(first % 3)};
  if (at.b < p.B && heads_of(at.op) == 0) advance(at);

  // ---------------- copies, kBwdStages passes ahead ----------------
  auto position = [&](const Unit& u) -> int {  // rot > 0
    if (p.rope.positions && u.b < p.B) return p.rope.positions[static_cast<long long>(u.b) * p.T + u.ti];
    return u.ti;
  };
  Unit ps = at, pn = at;  // the unit being copied and the one after it
  int p_row = 0, p_heads = 0, p_stage = 0, pos = 0, pos_ahead = 0;
  const uint16_t *p_g = nullptr, *p_x = nullptr;  // this lane's channels of its first row
  long long p_sh = 0;
  const long long g_set = static_cast<long long>(p.T) * D * ROWS;
  uint32_t live_bits = ~0u;  // bit s: the token of stage s has a row of the table
  if (p.rope.rot > 0) pos_ahead = position(ps);
  auto open = [&]() {  // addresses of unit ps; reads the position of the next
    if (ps.b >= p.B) return;
    p_heads = heads_of(ps.op);
    p_g = (ps.op == 0 ? p.gq : (ps.op == 1 ? p.gk : p.gv)) +
          ((static_cast<long long>(ps.b) * p_heads + t.sub) * p.T + ps.ti) * D + 8 * t.l;
    const Heads& x = ps.op == 0 ? p.q : p.k;
    const bool norm = ps.op == 0 ? p.rope.q_weight != nullptr : ps.op == 1 && p.rope.k_weight != nullptr;
    p_x = norm ? x.p + ps.b * x.sb + ps.ti * x.st + t.sub * x.sh + 8 * t.l : nullptr;
    p_sh = x.sh * ROWS;
    pos = pos_ahead;
    pn = ps;
    advance(pn);
    if (p.rope.rot > 0) pos_ahead = position(pn);
  };
  open();
  auto issue = [&]() {
    const int s = p_stage;
    p_stage = s + 1 == kBwdStages ? 0 : s + 1;
    if (ps.b < p.B) {
      const uint32_t dst = ring_addr + s * C::kStage;
      const bool more = p_row + PASS < p_heads;
      if (p_row + PASS <= p_heads) {
        const uint16_t* a = p_g;
#pragma unroll
        for (int u = 0; u < kBwdUnroll; ++u, a += g_set) copy16_async(dst + u * 512, a, true);
        p_g = a;
        if (p_x) {
          const uint16_t* c = p_x;
#pragma unroll
          for (int u = 0; u < kBwdUnroll; ++u, c += p_sh)
            copy16_async(dst + C::kHalf + u * 512, c, true);
          p_x = c;
        }
      } else {  // the unit's last rows: zeros behind them (from the address of a row it has)
#pragma unroll
        for (int u = 0; u < kBwdUnroll; ++u) {
          const int h = u * ROWS + t.sub, left = p_heads - p_row;
          const bool take = h < left;
          const long long set = take ? u : 0, back = take || t.sub < left ? 0 : t.sub;
          copy16_async(dst + u * 512, p_g + set * g_set - back * (g_set / ROWS), take);
          if (p_x) copy16_async(dst + C::kHalf + u * 512, p_x + set * p_sh - back * (p_sh / ROWS), take);
        }
      }
      if (p_row == 0 && p.rope.rot > 0) {
        const bool live = pos >= 0 && pos < p.rope.max_pos;
        if (!live && lane == 0) raise_flag(p.flags, DEVFLAG_BAD_POSITION);
        live_bits = (live_bits & ~(1u << s)) | (live ? 1u << s : 0u);
        if (4 * lane < p.rope.rot)
          copy16_async(dst + 2 * C::kHalf,
                       p.rope.cos_sin + static_cast<size_t>(live ? pos : 0) * p.rope.rot + 4 * lane, true);
      }
      p_row += PASS;
      if (!more) {
        p_row = 0;
        ps = pn;
        open();
      }
    }
    copy16_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kBwdStages; ++i) issue();

  // ---------------- pass by pass ----------------
  int left = 0, c_stage = 0;  // rows of the unit that are left; 0: a unit begins
  uint16_t* dx = nullptr;     // this lane's first channel of its first row
  long long dx_set = 0;
  while (at.b < p.B) {
    copy16_wait<kBwdStages - 1>();
    __syncwarp();
    const uint8_t* stage = ring + c_stage * C::kStage;
    const uint16_t* g = reinterpret_cast<const uint16_t*>(stage) + t.sub * D;
    const uint16_t* x = reinterpret_cast<const uint16_t*>(stage + C::kHalf) + t.sub * D;
    if (left == 0) {
      left = heads_of(at.op);
      const Heads& d = at.op == 0 ? p.dq : (at.op == 1 ? p.dk : p.dv);
      dx = d.p + at.b * d.sb + at.ti * d.st + t.sub * d.sh + (at.op == 2 ? 8 * t.l : t.ch.c0);
      dx_set = d.sh * ROWS;
      if (p.rope.rot > 0) {
        t.live = (live_bits >> c_stage) & 1u;
        float4 co = make_float4(1.f, 1.f, 1.f, 1.f), si = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t.ch.rotates && t.live) {
          const float* tab = reinterpret_cast<const float*>(stage + 2 * C::kHalf);
          co = *reinterpret_cast<const float4*>(tab + 4 * t.l);
          si = *reinterpret_cast<const float4*>(tab + p.rope.rot / 2 + 4 * t.l);
        }
        t.planes = Planes{{make_float2(co.x, co.y), make_float2(co.z, co.w)},
                          {make_float2(-si.x, -si.y), make_float2(-si.z, -si.w)}};
        if (!t.live) {  // a gradient through an unknown rotation is unknown
          const float nan = __int_as_float(0x7fc00000);
          dwq = dwk = Lane8{{{nan, nan}, {nan, nan}, {nan, nan}, {nan, nan}}};
        }
      }
    }
    // (sets past the last row compute with zeros: no branch keeps the sets apart)
    auto sets = [&](auto norm, const uint2(&w)[2], Lane8& dw) {
#pragma unroll(decltype(norm)::value ? 2 : 1)
      for (int u = 0; u < kBwdUnroll; ++u)
        norm_rope_bwd_set<D, INTERLEAVED, decltype(norm)::value>(
            t, g + u * ROWS * D, x + u * ROWS * D, w, dx + u * dx_set, u * ROWS + t.sub < left, dw);
    };
    if (at.op == 2) {
#pragma unroll
      for (int u = 0; u < kBwdUnroll; ++u)
        if (u * ROWS + t.sub < left)
          *reinterpret_cast<uint4*>(dx + u * dx_set) =
              *reinterpret_cast<const uint4*>(g + u * ROWS * D + 8 * t.l);
    } else if (at.op == 0) {
      if (p.rope.q_weight)
        sets(std::true_type{}, wq, dwq);
      else
        sets(std::false_type{}, wq, dwq);
    } else {
      if (p.rope.k_weight)
        sets(std::true_type{}, wk, dwk);
      else
        sets(std::false_type{}, wk, dwk);
    }
    left -= PASS;
    dx += kBwdUnroll * dx_set;
    if (left <= 0) {
      left = 0;
      advance(at);
    }
    __syncwarp();  // every lane has read the stage: the next pass may be copied over it
    c_stage = c_stage + 1 == kBwdStages ? 0 : c_stage + 1;
    issue();
  }
  if (p.part == nullptr) return;
  copy16_wait<0>();
  __syncthreads();  // the rings are done with
  float* red = reinterpret_cast<float*>(smem);  // [kBwdWarps * ROWS][2][D]
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int c = i < 4 ? t.ch.c0 + i : t.ch.c1 + i - 4;
    float* mine = red + (warp * ROWS + t.sub) * 2 * D + c;
    mine[0] = (i & 1) ? dwq.v[i / 2].y : dwq.v[i / 2].x;
    mine[D] = (i & 1) ? dwk.v[i / 2].y : dwk.v[i / 2].x;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += kBwdThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kBwdWarps * ROWS; ++i) s += red[i * 2 * D + e];
    p.part[static_cast<size_t>(blockIdx.x) * 2 * D + e] = s;
  }
}

// Adds the partials: 32 channels a CTA, 32 strided runs of partials each, a run's values all
// read at once (n = 0: zeros).
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float* part, int n, int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  // launched as a programmatic dependent: the partials are complete once this returns
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x * 32 + threadIdx.x;
  constexpr int RUN = (kBwdMaxGrid + 31) / 32;
  float v[RUN], s = 0.f;
#pragma unroll
  for (int k = 0; k < RUN; ++k) {
    const int i = threadIdx.y + 32 * k;
    v[k] = i < n ? part[static_cast<size_t>(i) * 2 * D + c] : 0.f;
  }
#pragma unroll
  for (int k = 0; k < RUN; ++k) s += v[k];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y != 0) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
  float* out = c < D ? dwq : dwk;
  if (out) out[c < D ? c : c - D] = s;
}

}  // namespace

int norm_rope_bwd_grid(int B, int T) {
  const long long want = (static_cast<long long>(B) * T + kBwdWarps - 1) / kBwdWarps;
  return static_cast<int>(want < kBwdMaxGrid ? want : kBwdMaxGrid);
}

size_t norm_rope_bwd_workspace_bytes(int B, int T, int D) {
  return static_cast<size_t>(norm_rope_bwd_grid(B, T)) * 2 * D * sizeof(float);
}

cudaError_t prepare_norm_rope() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void* fn, int bytes) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  set(reinterpret_cast<const void*>(norm_rope_bwd_kernel<64, false>), BwdShape<64>::kSmem);
  set(reinterpret_cast<const void*>(norm_rope_bwd_kernel<64, true>), BwdShape<64>::kSmem);
  set(reinterpret_cast<const void*>(norm_rope_bwd_kernel<128, false>), BwdShape<128>::kSmem);
  set(reinterpret_cast<const void*>(norm_rope_bwd_kernel<128, true>), BwdShape<128>::kSmem);
  return e;
}

cudaError_t launch_norm_rope_bwd(const NormRopeBwdParams& p, int D, cudaStream_t stream) {
  const int grid = norm_rope_bwd_grid(p.B, p.T);
  if (grid > 0 && p.nq + p.nk + p.nv > 0) {
    const bool il = p.rope.interleaved != 0;
    auto* kernel = D == 64 ? (il ? norm_rope_bwd_kernel<64, true> : norm_rope_bwd_kernel<64, false>)
                           : (il ? norm_rope_bwd_kernel<128, true> : norm_rope_bwd_kernel<128, false>);
    const cudaError_t e =
        launch_dependent(kernel, dim3(grid), dim3(kBwdThreads),
                         D == 64 ? BwdShape<64>::kSmem : BwdShape<128>::kSmem, stream, p);
    if (e != cudaSuccess) return e;
  }
  if (p.dwq == nullptr && p.dwk == nullptr) return cudaSuccess;
  return launch_dependent(norm_rope_dw_kernel, dim3(2 * D / 32), dim3(32, 32), 0, stream,
                          static_cast<const float*>(p.part), grid, D, p.dwq, p.dwk);
}

}  // namespace gbattn
