// kv4_decode.cu -- attention of single tokens and of short chunks against the 4-bit paged
// cache, sm_103a.
//
// For a query q and a token whose K group w has codes u_c = n_c + 8 and scale s_w, and
// whose V group has codes and scale t_w:
//   score  = scale * sum_w s_w sum_{c in w} q_c (u_c - 8)
//   O_c    = sum_tokens (p t_w) (u_c - 8) / sum_tokens p,    p = exp(score - max)
// so the codes go through the matrix units by themselves and the scales multiply the few
// score and probability values instead of the many cache values.
//
// A nibble becomes a matrix operand without any conversion of its bits, because the
// smallest floating-point numbers are equally spaced: a nibble alone in 16 bits, in
// either half of the low byte, is the fp16 number u 2^-24 or 16 u 2^-24 and the bf16 number
// u 2^-133 or 16 u 2^-133.  Two masks give four codes of a word, a shift by 8 the rest.
//   K: fp16 products take subnormal operands as they are.  The query's row is brought to
//      fp16 by a power of two that puts its largest element in [2^14, 2^15).  Channels whose
//      code sits in the upper half of a byte take q / 16.  fp16 goes down to 2^-24 and a bf16
//      has 8 bits, so elements down to 2^-27 of the largest (2^-31 without the / 16) are not
//      rounded, and smaller ones by at most 2^-35 (2^-39) of it, which an fp32 sum of the
//      row's products would not keep either.  (Rows below 2^-112 throughout lose more: they
//      are only brought up by 2^126.)  The products start from -8 sum q, which the same unit
//      computes once a piece.  The power of two goes into the softmax scale, and what that
//      does not hold as an fp32 (rows from about 2^93 on) into the scores (0.2 of 25 us).
//   V: p t needs the range of bf16, whose products do not take 2^-133; one fused
//      multiply-add on the pair makes it n / 64, exactly.
// Scores, softmax statistics and outputs are fp32; p t is rounded to bf16 for its product
// (2^-8 of itself at most, as the probabilities of the bf16 kernels are).  The running
// maximum only moves when it grows by more than 2^8, so outputs are rarely rescaled; p
// stays below 2^8.
//
// A token and KV head take 9 D / 8 bytes, read once.  The batch is one sequence of steps, 64
// tokens (4 blocks) of one (request, KV head) each, request-major; it is cut into equal
// ranges, and every warp streams a range by itself: lane j of the warp copies block j of a
// step, one untiled bulk copy of the whole chunk (codes and scales of K and V), into the
// warp's own ring in shared memory; the table entries of a step are read one step ahead of
// its copies.  The fragments of m16n8k16 come out of shared memory by plain loads in the
// order the format lays down.
//
// What bounds it: 64 requests of 512 to 8192 tokens, 12/2 heads, D 128 (80 MB, 11.8 us at
// the copy rate) take 25 us, one of 131000 tokens, 32/8 heads (151 MB, 22.2 us) 36 us.  The
// copies alone would take 12 and 30.  No pipe is full (issue slots 50 and 56 %, ALU 43 and
// 51 %, tensor 15 and 20 %): a step is one chain of loads, products, shuffles, exponentials
// and products, 3 us for the 12 warps an SM that 168 registers and two stages a warp leave
// room for, and too few warps to hide its latencies.  Set-up before the first copy lands
// is about 3 us, the merge kernel 4.  Steps of 2 blocks 27 and 41 us; 4 CTAs an SM
// (128 registers, spills) 31 and 47; V scales multiplied into transposed bf16 probabilities
// (22 of 230 instructions a block fewer, one more rounding) 25.4 and 37.2; V codes by 8-byte
// loads no change.
//
// A chunk of Tq tokens is the same computation with group * Tq query rows on every KV head
// ([Hq, Tq, D] keeps them together); row x sees the keys up to its own position.  Rows are
// taken 8 or 16 at a time, each such chunk of rows as a segment of its own (MULTI).
//
// The shortest range is one step, so that a small batch spreads over many SMs; ranges are
// dealt to the CTAs in turn for the same reason.  The piece of range k and segment s (both
// counted along the batch) is k + s: no two pieces share that number and those of one
// segment are consecutive, so the workspace holds ranges + segments pieces whatever the
// lengths.  The merge kernel gives every (request, query head) a CTA whose warps take its
// pieces in turn.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "norm_rope.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

constexpr int kBS = kPagedBlock;
constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStepBlocks = 4;  // blocks of one step: 64 tokens share a softmax update
// Deal::kDirect up to this max_seq_len.  Device time in us, direct / split, by max_seq_len
// (lengths from half of it):
//   5 x 16/1 heads, D 64:     256: 3.7 / 7.3    512: 4.8 / 7.4    768: 6.1 / 7.4    1024: 7.5 / 7.3
//   1 x 12/2, D 128:          256: 3.7 / 6.6    512: 5.2 / 7.0    768: 5.0 / 7.1    1024: 6.7 / 7.2
//   64 x 12/2, D 128:         256: 5.7 / 8.8    512: 8.3 / 10.0   768: 10.4 / 10.1  1024: 13.2 / 10.2
//   200 x 8/2, D 128:         256: 6.5 / 11.0   512: 9.6 / 14.5   768: 12.4 / 15.9  1024: 15.1 / 18.2
//   64 x 32/8, D 128:         256: 8.4 / 11.1   512: 12.6 / 15.4  768: 15.8 / 18.6  1024: 19.3 / 21.1
// An eager call adds 0.2 to 2 us to either.  Batches of about one CTA an SM are the
// exception above 700 tokens: their few steps a warp are a longer chain than the split's.
constexpr int kDirectMaxLen = 1024;
constexpr float kRescaleLog2 = 8.f;  // move the running max only if it grows by > 2^8

// Ring depth and CTAs per SM by query tiles (NQT = 1: groups of up to 8 query heads,
// 2: up to 16, which needs the registers of two CTAs).
template <int D, int NQT>
struct Shape {
  static constexpr int kStageBytes = kStepBlocks * Kv4<D>::kChunk;
  static constexpr int kCtasPerSm = NQT == 1 ? 3 : 2;
  static constexpr int kStages = (D == 64 ? 2 : 1) * (NQT == 1 ? 2 : 3);
  static constexpr int kOffBar = kWarps * kStages * kStageBytes;
  static constexpr int kOffAbort = kOffBar + kWarps * kStages * 8;
  static constexpr int kOffBoost = kOffAbort + kWarps * 4;  // [kWarps][8 NQT] floats
  static constexpr int kSmem = kOffBoost + kWarps * 8 * NQT * 4 + 128;  // slack for 128-byte alignment
};

// D = A * B + C (C may be D), m16n8k16, fp16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
        "f"(c3));
}

// D = A * B + D, m16n8k16, bf16 inputs, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit values held across the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

constexpr uint32_t kLowNibbles = 0x000f000fu, kHighNibbles = 0x00f000f0u;

// The masked codes of a pair, u 2^-133 or 16 u 2^-133, as bf16 (u - 8) / 64.
__device__ __forceinline__ uint32_t centre(uint32_t codes, uint32_t factor) {
  const uint32_t off = 0xbe00be00u;  // -2^-3
  uint32_t y;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(codes), "r"(factor), "r"(off));
  return y;
}
constexpr uint32_t kLowFactor = 0x7f007f00u, kHighFactor = 0x7d007d00u;  // 2^127, 2^123

// Two fp32 as an fp16 pair: lo -> bits 0-15.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 2^x as an fp32, -126 <= x <= 127.
__device__ __forceinline__ float pow2(int x) { return __int_as_float((127 + x) << 23); }

// Token of a 16-token block that row `row` of a score tile holds.  Neighbouring rows are
// swapped in every other pair, so that both the K loads (rows 2 a, 2 a + 1 together) and
// the V loads (rows 0, 2, 4, 6 together) meet tokens of either parity, i.e. both halves
// of the shared-memory banks.
__device__ __forceinline__ int token_of_row(int row) { return row ^ ((row >> 1) & 1); }

template <int N>
__device__ __forceinline__ void lds(const uint8_t* p, uint32_t (&r)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "4, 8 or 16 bytes");
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    r[0] = v.x, r[1] = v.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// Scale w of a row's packed scales.
template <int N>
__device__ __forceinline__ float scale_of(const uint32_t (&r)[N], int w) {
  return (w & 1) ? bf16_hi(r[w >> 1]) : bf16_lo(r[w >> 1]);
}

// Blocks per KV head of a request of L tokens; 0 for a length outside its bounds (the
// merge kernel reports that request).
__device__ __forceinline__ int blocks_of(const Kv4DecodeParams& p, int L) {
  return (L < 0 || L > p.max_seq_len || L > p.max_blocks * kBS) ? 0 : (L + kBS - 1) / kBS;
}

__device__ __forceinline__ int steps_of(int blocks) { return (blocks + kStepBlocks - 1) / kStepBlocks; }

// A step of the batch: step i of request r, segment h (a KV head, or MULTI a KV head and a
// chunk of rows), which has nb blocks.
struct Step {
  int r, h, i, nb;
  __device__ int blocks() const { return min(kStepBlocks, nb - i * kStepBlocks); }
  __device__ bool last() const { return (i + 1) * kStepBlocks >= nb; }
};

// The next step of the batch; r stops at S, should the lengths have changed.
__device__ __forceinline__ void advance(Step& s, const Kv4DecodeParams& p) {
  if (!s.last()) {
    ++s.i;
    return;
  }
  s.i = 0;
  if (++s.h < p.segs) return;
  s.h = 0;
  s.nb = 0;
  while (s.nb == 0 && ++s.r < p.S) s.nb = blocks_of(p, p.seq_lens[s.r]);
}

// How the work is dealt.  kSplit and kMulti (the rows of a chunk in several segments): the
// batch's steps in equal ranges, a merge kernel after.  kDirect, for short caches: a CTA a
// segment, whose warps take its steps in turn and join their results in shared memory; no
// workspace and one launch.
enum class Deal { kSplit, kMulti, kDirect };

template <int D, int NQT, Deal DEAL>
__global__ void __launch_bounds__(kThreads, Shape<D, NQT>::kCtasPerSm)
    kv4_decode_split_kernel(const uint8_t* __restrict__ pool, const Kv4DecodeParams p) {
  using F = Kv4<D>;
  using C = Shape<D, NQT>;
  constexpr bool MULTI = DEAL == Deal::kMulti, DIRECT = DEAL == Deal::kDirect;
  constexpr int G = F::kGroups;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 127u) & ~127u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* ring = smem + warp * C::kStages * C::kStageBytes;
  const uint32_t ring_addr = sbase + warp * C::kStages * C::kStageBytes;
  const uint32_t bars = sbase + C::kOffBar + warp * C::kStages * 8;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::kOffAbort) + warp;
  float* boost = reinterpret_cast<float*>(smem + C::kOffBoost) + warp * 8 * NQT;

  // the merge kernel (or what else follows as a programmatic dependent) may be scheduled
  // now; it waits for this grid's results
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (lane == 0) {
    for (int s = 0; s < C::kStages; ++s) mbar_init(bars + 8 * s, 1);
    *abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  __syncwarp();
  // the preceding kernel's writes (an append's) are complete and visible past this point
  asm volatile("griddepcontrol.wait;" ::: "memory");

  Step at{0, 0, 0, 0};  // this warp's first step, and how many steps it takes
  int n_w = 0, k_w = 0;
  if constexpr (DIRECT) {
    at.r = blockIdx.x / p.segs;
    at.h = blockIdx.x - at.r * p.segs;
    at.i = warp;
    at.nb = blocks_of(p, p.seq_lens[at.r]);
    n_w = (steps_of(at.nb) - warp + kWarps - 1) / kWarps;
  } else {
    // ---------------- plan: total steps, range count, this warp's range ----------------
    // (128 requests a round: a lane's four lengths are read at once)
    int total = 0, nb4[4];
    auto read4 = [&](int r0) {
      int L[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) L[i] = r0 + 32 * i + lane < p.S ? p.seq_lens[r0 + 32 * i + lane] : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) nb4[i] = blocks_of(p, L[i]);
    };
    for (int r0 = 0; r0 < p.S; r0 += 128) {
      read4(r0);
#pragma unroll
      for (int i = 0; i < 4; ++i) total += steps_of(nb4[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    total *= p.segs;  // below 2^31 for every length within max_seq_len
    const int W = min(static_cast<int>(gridDim.x) * kWarps, total);
    k_w = warp * gridDim.x + blockIdx.x;
    if (k_w >= W) return;  // warps are independent: no barrier of the CTA follows
    const int share = total / W, extra = total - share * W;  // the first `extra` take one more
    const int lo = k_w * share + min(k_w, extra);
    n_w = share + (k_w < extra ? 1 : 0);
    {
      int before = 0;  // steps of requests r0 - 1 and earlier
      bool found = false;
      for (int r0 = 0; r0 < p.S && !found; r0 += 32) {
        if (p.S > 128 && r0 % 128 == 0) read4(r0);
        const int i = r0 / 32 % 4;
        const int nb = i < 2 ? (i == 0 ? nb4[0] : nb4[1]) : (i == 2 ? nb4[2] : nb4[3]);
        const int own = steps_of(nb) * p.segs;
        int incl = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        incl += before;
        const unsigned hit = __ballot_sync(0xffffffffu, incl - own <= lo && lo < incl);
        if (hit) {
          found = true;
          const int src = __ffs(hit) - 1;
          const int rest = lo - __shfl_sync(0xffffffffu, incl - own, src);
          at.nb = __shfl_sync(0xffffffffu, nb, src);
          at.r = r0 + src;
          at.h = rest / steps_of(at.nb);
          at.i = rest - at.h * steps_of(at.nb);
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
      }
      if (!found) return;  // lengths changed under the kernel
    }
  }
  auto next = [&](Step& st) {
    if constexpr (DIRECT)
      st.i += kWarps;
    else
      advance(st, p);
  };

  // ---------------- copies: one step ahead in table entries, kStages in data ----------------
  Step ps = at;
  int p_left = n_w, issued = 0, p_stage = 0;
  const uint64_t policy = l2_policy_evict_first();  // every cache byte is read once
  auto kv_head = [&](int h) { return MULTI ? h / p.chunks : h; };
  auto entry = [&]() -> int {
    return lane < ps.blocks()
               ? p.block_table[static_cast<size_t>(ps.r) * p.max_blocks + ps.i * kStepBlocks + lane]
               : 0;
  };
  int phys = p_left > 0 ? entry() : 0;
  uint32_t stage_bad = 0;  // bit s: stage s holds a block the table could not translate
  auto issue = [&]() {     // copies step ps, then reads the table entries of the next one
    const int s = p_stage, n = ps.blocks();
    const bool bad = lane < n && (phys < 0 || phys >= p.num_pool_blocks);
    if (bad) raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
    stage_bad = (stage_bad & ~(1u << s)) | (__any_sync(0xffffffffu, bad) ? 1u << s : 0u);
    if (!(p.withhold_copy && issued == 0)) {  // test hook: the first step never arrives
      if (lane == 0) mbar_arrive_expect_tx(bars + 8 * s, n * F::kChunk);
      __syncwarp();
      if (lane < n)
        bulk_load_hint(ring_addr + s * C::kStageBytes + lane * F::kChunk,
                       pool + (static_cast<size_t>(bad ? 0 : phys) * p.Hkv + kv_head(ps.h)) * F::kChunk,
                       F::kChunk, bars + 8 * s, policy);
    }
    ++issued;
    p_stage = s + 1 == C::kStages ? 0 : s + 1;
    if (--p_left > 0) {
      next(ps);
      if (ps.r >= p.S)
        p_left = 0;  // lengths changed under the kernel: nothing valid to read
      else
        phys = entry();
    }
  };
#pragma unroll 1
  for (int i = 0; i < C::kStages && p_left > 0; ++i) issue();

  // ---------------- the range, step by step ----------------
  const int g = lane >> 2, t4 = lane & 3;
  int n_rows = p.rows;               // query rows of the segment
  const int row0 = token_of_row(g);  // rows g and g + 8 of a score tile: tokens row0 (+ 8)
  uint32_t qb[D / 16][NQT][2];       // Q^T fragments (fp16) in the order of the K codes
  float q8[G][NQT][2];               // -8 sum of q over group w, queries 2 t4 (+ 1)
  float sl2[NQT][2], sl[NQT][2];     // softmax scale (times log2 e) over the query's 2^x
  bool boosted = false;              // some query's scores take a factor (boost) first
  float m_q[NQT][2], l_q[NQT][2];
  float acc[D / 16][NQT][4];         // O^T / 64: channels 32 w + 4 g + 2 x (+ 1) of tile 2 w + x
  Step c = at;
  int c_left = n_w, taken = 0, c_stage = 0, L = 0;
  uint32_t phase = 0;
  bool pbad = false, ok = true;

  auto begin_piece = [&]() {
    L = p.seq_lens[c.r];
    pbad = false;
    if (!DIRECT && c.i == 0 && lane == 0) p.seg_first[c.r * p.segs + c.h] = k_w;
    size_t q0 = static_cast<size_t>(c.r) * p.Hkv * p.rows + static_cast<size_t>(c.h) * p.rows;
    if constexpr (MULTI) {
      const int h = c.h / p.chunks, x0 = (c.h - h * p.chunks) * (8 * NQT);
      n_rows = min(8 * NQT, p.rows - x0);
      q0 = (static_cast<size_t>(c.r) * p.Hkv + h) * p.rows + x0;
    }
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + q0 * D;
    // A fragment of -8 in both forms of a code
    const uint32_t minus8[4] = {0x80088008u, 0x80088008u, 0x80808080u, 0x80808080u};
    bool big_scale = false;
#pragma unroll
    for (int nt = 0; nt < NQT; ++nt) {
      const int row = 8 * nt + g;
      uint4 x[G];
      uint32_t big = 0;  // largest magnitude of the row, as bf16 bits in either half
#pragma unroll
      for (int w = 0; w < G; ++w) {
        x[w] = make_uint4(0, 0, 0, 0);
        if (row < n_rows) x[w] = *reinterpret_cast<const uint4*>(q + row * D + 32 * w + 8 * t4);
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(x[w].x & 0x7fff7fffu, x[w].y & 0x7fff7fffu),
                                     __vmaxu2(x[w].z & 0x7fff7fffu, x[w].w & 0x7fff7fffu)));
      }
      big = max(big & 0xffffu, big >> 16);
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // q = q' 2^(e - 14): e the exponent of the largest element (128: an infinity or NaN),
      // kept where the factor is a normal number
      const int e = max(static_cast<int>(big >> 7) - 127, -112);
      const float f0 = pow2(14 - e), f1 = f0 * 0.0625f;
#pragma unroll
      for (int w = 0; w < G; ++w) {
        // masks of a word give channels 0, 4 (low) and 1, 5 (high); shifted by 8: 2, 6 and 3, 7
        qb[2 * w][nt][0] = pack_f16x2(bf16_lo(x[w].x) * f0, bf16_lo(x[w].z) * f0);
        qb[2 * w][nt][1] = pack_f16x2(bf16_hi(x[w].x) * f1, bf16_hi(x[w].z) * f1);
        qb[2 * w + 1][nt][0] = pack_f16x2(bf16_lo(x[w].y) * f0, bf16_lo(x[w].w) * f0);
        qb[2 * w + 1][nt][1] = pack_f16x2(bf16_hi(x[w].y) * f1, bf16_hi(x[w].w) * f1);
        float d[4];
        mma_f16(d, minus8, qb[2 * w][nt][0], qb[2 * w][nt][1], 0.f, 0.f, 0.f, 0.f);
        mma_f16(d, minus8, qb[2 * w + 1][nt][0], qb[2 * w + 1][nt][1], d[0], d[1], d[2], d[3]);
        q8[w][nt][0] = d[0];
        q8[w][nt][1] = d[1];
      }
#pragma unroll
      for (int x2 = 0; x2 < 2; ++x2) {
        // lane 4 k holds the exponent of query k: this lane's columns are 2 t4 and 2 t4 + 1
        const int eq = __shfl_sync(0xffffffffu, e, 4 * (2 * t4 + x2));
        // scale 2^(eq + 24 - 14), in two steps as the power alone may not be a number, and
        // what it has above 2^100 as a factor of the scores
        const int sx = static_cast<int>(__float_as_uint(p.scale_log2) >> 23) - 127;
        const int over = min(max(eq + 10 + sx - 100, 0), 126), x = eq + 10 - over;
        const float fa = pow2(x >> 1), fb = pow2(x - (x >> 1));
        sl[nt][x2] = p.scale * fa * fb;
        sl2[nt][x2] = fmaxf(p.scale_log2 * fa * fb, 1.17549435e-38f);  // (0 times the first -inf: NaN)
        big_scale |= over > 0;
        if (g == 0) boost[8 * nt + 2 * t4 + x2] = pow2(over);
        m_q[nt][x2] = -INFINITY;
        l_q[nt][x2] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
        acc[j][nt][0] = acc[j][nt][1] = acc[j][nt][2] = acc[j][nt][3] = 0.f;
    }
    boosted = __any_sync(0xffffffffu, big_scale);
    __syncwarp();
  };
  begin_piece();  // (DIRECT: also by a warp without a step, whose sums stay empty)

  while (c_left > 0) {
    const int s = c_stage;
    if (!mbar_wait_warp(bars + 8 * s, phase, abort, p.flags, p.wait_limit_ns)) {
      ok = false;
      break;
    }
    pbad |= (stage_bad >> s) & 1u;
    const uint8_t* stage = ring + s * C::kStageBytes;
    // Valid tokens of the step.  The blocks past them are computed with whatever the stage
    // holds (codes are finite whatever their bits) and masked with the tail.
    const int here = L - c.i * (kBS * kStepBlocks);  // keys from the step's first on
    const int n_tok = min(kBS * kStepBlocks, here);

    // ---- S^T = K Q^T, group by group ----
    float sc[kStepBlocks][NQT][4];
#pragma unroll
    for (int j = 0; j < kStepBlocks; ++j) {
      const uint8_t* blk = stage + j * F::kChunk;
      uint32_t k0[G], k1[G], s0[G / 2], s1[G / 2];
      lds(blk + F::kOffKCodes + row0 * F::kCodeRow + t4 * (4 * G), k0);
      lds(blk + F::kOffKCodes + (row0 + 8) * F::kCodeRow + t4 * (4 * G), k1);
      lds(blk + F::kOffKScales + row0 * F::kScaleRow, s0);
      lds(blk + F::kOffKScales + (row0 + 8) * F::kScaleRow, s1);
#pragma unroll
      for (int w = 0; w < G; ++w) {
        const uint32_t h0 = k0[w] >> 8, h1 = k1[w] >> 8;
        const uint32_t a0[4] = {k0[w] & kLowNibbles, k1[w] & kLowNibbles, k0[w] & kHighNibbles,
                                k1[w] & kHighNibbles};
        const uint32_t a1[4] = {h0 & kLowNibbles, h1 & kLowNibbles, h0 & kHighNibbles,
                                h1 & kHighNibbles};
        const float f0 = scale_of(s0, w), f1 = scale_of(s1, w);
#pragma unroll
        for (int nt = 0; nt < NQT; ++nt) {
          float d[4];
          const float c0 = q8[w][nt][0], c1 = q8[w][nt][1];
          mma_f16(d, a0, qb[2 * w][nt][0], qb[2 * w][nt][1], c0, c1, c0, c1);
          mma_f16(d, a1, qb[2 * w + 1][nt][0], qb[2 * w + 1][nt][1], d[0], d[1], d[2], d[3]);
          if (w == 0) {
            sc[j][nt][0] = f0 * d[0];
            sc[j][nt][1] = f0 * d[1];
            sc[j][nt][2] = f1 * d[2];
            sc[j][nt][3] = f1 * d[3];
          } else {
            sc[j][nt][0] = fmaf(f0, d[0], sc[j][nt][0]);
            sc[j][nt][1] = fmaf(f0, d[1], sc[j][nt][1]);
            sc[j][nt][2] = fmaf(f1, d[2], sc[j][nt][2]);
            sc[j][nt][3] = fmaf(f1, d[3], sc[j][nt][3]);
          }
        }
      }
    }
    if (boosted) {
#pragma unroll
      for (int nt = 0; nt < NQT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float f = boost[8 * nt + 2 * t4 + e];
#pragma unroll
          for (int j = 0; j < kStepBlocks; ++j) {
            sc[j][nt][e] *= f;
            sc[j][nt][2 + e] *= f;
          }
        }
      }
    }
    // MULTI, causal: row x sees the keys before its own position and its own
    const int hidden = MULTI && p.causal ? p.Tq - 1 : 0;  // keys that row 0 does not see
    const bool tail = here - hidden < kBS * kStepBlocks;
    if (MULTI && tail) {
      const int x0 = (c.h % p.chunks) * (8 * NQT) + 2 * t4;
#pragma unroll
      for (int nt = 0; nt < NQT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int n = min(here, here - hidden + (p.causal ? (x0 + 8 * nt + e) % p.Tq : 0));
#pragma unroll
          for (int j = 0; j < kStepBlocks; ++j) {
            if (kBS * j + row0 >= n) sc[j][nt][e] = -INFINITY;
            if (kBS * j + row0 + 8 >= n) sc[j][nt][2 + e] = -INFINITY;
          }
        }
      }
    } else if (tail) {  // tokens past the end: their codes and scales may be anything
#pragma unroll
      for (int j = 0; j < kStepBlocks; ++j) {
        const bool in0 = kBS * j + row0 < n_tok, in1 = kBS * j + row0 + 8 < n_tok;
#pragma unroll
        for (int nt = 0; nt < NQT; ++nt) {
          if (!in0) sc[j][nt][0] = sc[j][nt][1] = -INFINITY;
          if (!in1) sc[j][nt][2] = sc[j][nt][3] = -INFINITY;
        }
      }
    }

    // ---- softmax update (one per step) ----
    float al[NQT][2];
    bool grown = false;
#pragma unroll
    for (int nt = 0; nt < NQT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float bm = fmaxf(sc[0][nt][e], sc[0][nt][2 + e]);
#pragma unroll
        for (int j = 1; j < kStepBlocks; ++j) bm = fmax3(bm, sc[j][nt][e], sc[j][nt][2 + e]);
        // lanes with the same t4 hold the step's other tokens
        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 4));
        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 8));
        bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, 16));
        // (finite from the first step on: every step has a valid token, but MULTI rows may
        // not see it)
        const bool grow = (bm - m_q[nt][e]) * sl2[nt][e] > kRescaleLog2;
        al[nt][e] = grow ? ex2((m_q[nt][e] - bm) * sl2[nt][e]) : 1.f;
        m_q[nt][e] = grow ? bm : m_q[nt][e];
        grown |= grow;
        const float ms = MULTI && m_q[nt][e] == -INFINITY ? 0.f : m_q[nt][e] * sl2[nt][e];
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < kStepBlocks; ++j) {
#pragma unroll
          for (int x = e; x < 4; x += 2) {
            sc[j][nt][x] = ex2(fmaf(sc[j][nt][x], sl2[nt][e], -ms));
            sum += sc[j][nt][x];
          }
        }
        l_q[nt][e] = l_q[nt][e] * al[nt][e] + sum;
      }
    }
    if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int nt = 0; nt < NQT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[j][nt][x] *= al[nt][x & 1];
    }

    // ---- O^T += V^T (P t)^T, two groups (one word of V codes) at a time ----
#pragma unroll
    for (int j = 0; j < kStepBlocks; ++j) {
      const uint8_t* blk = stage + j * F::kChunk;
      const int ta = token_of_row(2 * t4), tb = token_of_row(2 * t4 + 1);
#pragma unroll
      for (int u = 0; u < G / 2; ++u) {
        // (p t)^T fragments of groups 2 u and 2 u + 1
        const uint8_t* sv = blk + F::kOffVScales + 4 * u;
        uint32_t t0 = *reinterpret_cast<const uint32_t*>(sv + row0 * F::kScaleRow);
        uint32_t t1 = *reinterpret_cast<const uint32_t*>(sv + (row0 + 8) * F::kScaleRow);
        if (tail) {  // p is 0 there, but 0 * NaN is not
          if (kBS * j + row0 >= n_tok) t0 = 0;
          if (kBS * j + row0 + 8 >= n_tok) t1 = 0;
        }
        // V^T fragments: channels 4 g .. of each group, score rows 2 t4, 2 t4 + 1 (+ 8)
        const uint8_t* v = blk + F::kOffVCodes + g * (2 * G) + 4 * u;
        const uint32_t va = *reinterpret_cast<const uint32_t*>(v + ta * F::kCodeRow);
        const uint32_t vb = *reinterpret_cast<const uint32_t*>(v + tb * F::kCodeRow);
        const uint32_t vc = *reinterpret_cast<const uint32_t*>(v + (ta + 8) * F::kCodeRow);
        const uint32_t vd = *reinterpret_cast<const uint32_t*>(v + (tb + 8) * F::kCodeRow);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const float f0 = x ? bf16_hi(t0) : bf16_lo(t0), f1 = x ? bf16_hi(t1) : bf16_lo(t1);
          uint32_t pb[NQT][2];
#pragma unroll
          for (int nt = 0; nt < NQT; ++nt) {
            pb[nt][0] = transpose8x8(pack_bf16x2(sc[j][nt][0] * f0, sc[j][nt][1] * f0));
            pb[nt][1] = transpose8x8(pack_bf16x2(sc[j][nt][2] * f1, sc[j][nt][3] * f1));
          }
          const uint32_t ab = __byte_perm(va, vb, x ? 0x7632 : 0x5410);
          const uint32_t cd = __byte_perm(vc, vd, x ? 0x7632 : 0x5410);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t ab8 = y ? ab >> 8 : ab, cd8 = y ? cd >> 8 : cd;
            const uint32_t a[4] = {centre(ab8 & kLowNibbles, kLowFactor),
                                   centre(ab8 & kHighNibbles, kHighFactor),
                                   centre(cd8 & kLowNibbles, kLowFactor),
                                   centre(cd8 & kHighNibbles, kHighFactor)};
#pragma unroll
            for (int nt = 0; nt < NQT; ++nt)
              mma_bf16(acc[2 * (2 * u + x) + y][nt], a, pb[nt][0], pb[nt][1]);
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage: the next step may be copied over it
    ++taken;
    if (++c_stage == C::kStages) {
      c_stage = 0;
      phase ^= 1;
    }
    if (p_left > 0) issue();

    --c_left;
    if constexpr (DIRECT) {
      c.i += kWarps;
      continue;
    }
    if (!c.last() && c_left > 0) {
      ++c.i;
      continue;
    }
    // ---- the piece ends: write its normalised O and LSE ----
    {
      const float nan = __int_as_float(0x7fc00000);
      const int seg = c.r * p.segs + c.h, piece = k_w + seg;
      if (piece < p.max_pieces) {
#pragma unroll
        for (int nt = 0; nt < NQT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float lsum = l_q[nt][e];
            lsum += __shfl_xor_sync(0xffffffffu, lsum, 4);
            lsum += __shfl_xor_sync(0xffffffffu, lsum, 8);
            lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);
            const int q = 8 * nt + 2 * t4 + e;
            if (q >= n_rows) continue;
            const bool none = MULTI && lsum == 0.f;  // no key of the piece is visible
            const float inv = pbad ? nan : (none ? 0.f : 64.f / lsum);
            const size_t base = static_cast<size_t>(piece) * p.piece_rows + q;
            float* dst = p.part_o + base * D + 4 * g;
#pragma unroll
            for (int w = 0; w < G; ++w)
              *reinterpret_cast<float4*>(dst + 32 * w) =
                  make_float4(acc[2 * w][nt][e] * inv, acc[2 * w][nt][2 + e] * inv,
                              acc[2 * w + 1][nt][e] * inv, acc[2 * w + 1][nt][2 + e] * inv);
            if (g == 0)
              p.part_lse[base] =
                  pbad ? nan : (none ? -INFINITY : m_q[nt][e] * sl[nt][e] + logf(lsum));
          }
        }
        if (c.last() && lane == 0) p.seg_last[seg] = k_w;
      }
    }
    if (c_left == 0) break;
    // the range continues in the next segment
    advance(c, p);
    if (c.r >= p.S) break;  // lengths changed under the kernel: nothing valid to read
    begin_piece();
  }
  // Copies still in flight land before the CTA's shared memory goes away.
  if (!ok || taken < issued)
    for (int i = taken; i < issued; ++i)
      if (!(p.withhold_copy && i == 0))
        mbar_wait_quiet(bars + 8 * (i % C::kStages), (i / C::kStages) & 1, 500000000ull);
  if constexpr (DIRECT) {
    // ---- join the warps' sums; the rings are done with ----
    constexpr int R = 8 * NQT;
    float* po = reinterpret_cast<float*>(smem);       // [kWarps][R][D] O / 64, not normalised
    float* pm = po + kWarps * R * D;                  // [kWarps][R] maximum, in log2 units
    float* pl = pm + kWarps * R;                      // [kWarps][R] sum
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NQT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float lsum = l_q[nt][e];
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 4);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 8);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);
        const int q = warp * R + 8 * nt + 2 * t4 + e;
#pragma unroll
        for (int w = 0; w < G; ++w)
          *reinterpret_cast<float4*>(po + q * D + 4 * g + 32 * w) =
              make_float4(acc[2 * w][nt][e], acc[2 * w][nt][2 + e], acc[2 * w + 1][nt][e],
                          acc[2 * w + 1][nt][2 + e]);
        if (g == 0) {
          // a block that the table could not translate makes the whole request NaN
          pm[q] = m_q[nt][e] == -INFINITY ? -INFINITY : m_q[nt][e] * sl2[nt][e];
          pl[q] = pbad ? __int_as_float(0x7fc00000) : lsum;
        }
      }
    }
    __syncthreads();
    const bool bad_len = at.nb == 0 && L != 0;
    if (bad_len && threadIdx.x == 0) raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
    constexpr int TPR = D / 2;  // threads of a row, two channels each
    const size_t row0_out = (static_cast<size_t>(at.r) * p.segs + at.h) * p.rows;
    for (int q = threadIdx.x / TPR; q < p.rows; q += kThreads / TPR) {
      const int d = threadIdx.x % TPR * 2;
      float M = pm[q];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) M = fmaxf(M, pm[w * R + q]);
      const float Ms = M == -INFINITY ? 0.f : M;
      float tot = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(pm[w * R + q] - Ms);
        const float2 v = *reinterpret_cast<const float2*>(po + (w * R + q) * D + d);
        tot = fmaf(f, pl[w * R + q], tot);
        x0 = fmaf(f, v.x, x0);
        x1 = fmaf(f, v.y, x1);
      }
      const float inv = tot == 0.f ? 0.f : 64.f / tot;
      float lse = Ms * 0.6931471805599453f + logf(tot);  // (log 0 = -inf: an empty cache)
      x0 *= inv;
      x1 *= inv;
      if (bad_len) x0 = x1 = lse = __int_as_float(0x7fc00000);
      reinterpret_cast<uint32_t*>(p.o)[((row0_out + q) * D + d) / 2] = pack_bf16x2(x0, x1);
      if (p.lse != nullptr && d == 0) p.lse[row0_out + q] = lse;
    }
  }
}

// LSE = M + ln sum_j e^{LSE_j - M}, O = sum_j e^{LSE_j - LSE} O_j over the pieces of one
// (request, query head): a CTA, whose MW warps take every MW-th piece, four of them in
// flight at a time, and are joined in shared memory.  A NaN of a piece goes through.
//
// The whole takes some 4 us, more than its two round trips of reads: a first run of the code
// is slow.  With many warps a head, i.e. few CTAs, each goes through it once over no pieces
// before it waits for the split kernel, which then still runs (36.6 -> 35.9 us a call on
// 131000 tokens, 19.1 -> 18.5 on 40000; the 768 CTAs of 64 requests would take issue slots
// from the split kernel: 25.0 -> 25.3).  It does not let the next call's split kernel in
// early: that one takes the room its own CTAs need (64 requests in a row 24.6 -> 29.0 us).
template <int D, int MW>
__global__ void __launch_bounds__(MW * 32) kv4_decode_merge_kernel(const Kv4DecodeParams p) {
  constexpr int PER = D / 32;  // dims per lane
  constexpr float kLog2e = 1.4426950408889634f;
  __shared__ float part[MW][D];
  __shared__ float part_m[MW], part_sum[MW];
  // the CTA's row: row x of KV head kvh of request r
  const int kv = blockIdx.x / p.rows, x = blockIdx.x - kv * p.rows;
  const int r = kv / p.Hkv, kvh = kv - r * p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunk = x / p.piece_rows;
  const int seg = r * p.segs + kvh * p.chunks + chunk;
#pragma unroll 1
  for (int pass = MW > 4 ? 0 : 1; pass < 2; ++pass) {
    int L = 0, k0 = 0, k1 = -1;
    if (pass == 1) {
      // launched as a programmatic dependent: the split kernel's results are complete and
      // visible once this returns
      asm volatile("griddepcontrol.wait;" ::: "memory");
      L = p.seq_lens[r];
      k0 = p.seg_first[seg];
      k1 = p.seg_last[seg];
    }
    // (the split kernel has noted the ranges of every valid nonempty request; the check keeps
    // every read in bounds should the lengths have changed between the two kernels)
    const bool good = blocks_of(p, L) > 0 && k0 >= 0 && k0 <= k1 && k1 + seg < p.max_pieces;
    const bool bad = L != 0 && !good;
    const int n = good ? k1 - k0 + 1 : 0;
    const size_t base =
        good ? static_cast<size_t>(k0 + seg) * p.piece_rows + (x - chunk * p.piece_rows) : 0;
    const float* pl = p.part_lse + base;
    const float* po = p.part_o + base * D + lane * PER;

    float m = -INFINITY, sum = 0.f, o[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) o[i] = 0.f;
    // (a first round without pieces is taken too, for the reason above)
    for (int j0 = warp; j0 < n || (pass == 0 && j0 == warp); j0 += 4 * MW) {
      float lse[4], v[4][PER];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int j = j0 + s * MW;
        lse[s] = -INFINITY;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[s][i] = 0.f;
        if (j < n) {
          lse[s] = pl[static_cast<size_t>(j) * p.piece_rows];
          const float* src = po + static_cast<size_t>(j) * p.piece_rows * D;
          if constexpr (PER == 4) {
            const float4 x = *reinterpret_cast<const float4*>(src);
            v[s][0] = x.x, v[s][1] = x.y, v[s][2] = x.z, v[s][3] = x.w;
          } else {
            const float2 x = *reinterpret_cast<const float2*>(src);
            v[s][0] = x.x, v[s][1] = x.y;
          }
        }
      }
      const float mn = fmaxf(fmaxf(m, lse[0]), fmax3(lse[1], lse[2], lse[3]));
      const float ms = mn == -INFINITY ? 0.f : mn;  // (all four NaN, or no piece)
      const float al = ex2((m - ms) * kLog2e);
      m = mn;
      sum *= al;
#pragma unroll
      for (int i = 0; i < PER; ++i) o[i] *= al;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const float w = ex2((lse[s] - ms) * kLog2e);
        sum += w;
#pragma unroll
        for (int i = 0; i < PER; ++i) o[i] = fmaf(w, v[s][i], o[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) part[warp][lane * PER + i] = o[i];
    if (lane == 0) {
      part_m[warp] = m;
      part_sum[warp] = sum;
    }
    __syncthreads();
    if (threadIdx.x < D / 2) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < MW; ++w) M = fmaxf(M, part_m[w]);
      const float Ms = M == -INFINITY ? 0.f : M;
      float tot = 0.f, x0 = 0.f, x1 = 0.f;
#pragma unroll
      for (int w = 0; w < MW; ++w) {
        const float f = ex2((part_m[w] - Ms) * kLog2e);
        tot = fmaf(f, part_sum[w], tot);
        x0 = fmaf(f, part[w][2 * threadIdx.x], x0);
        x1 = fmaf(f, part[w][2 * threadIdx.x + 1], x1);
      }
      float lse_out = Ms + logf(tot);
      const float inv = tot == 0.f ? 0.f : 1.f / tot;  // (no key is visible to the row)
      x0 *= inv;
      x1 *= inv;
      if (bad) {
        if (threadIdx.x == 0) raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
        x0 = x1 = lse_out = __int_as_float(0x7fc00000);
      }
      if (pass == 1) {
        reinterpret_cast<uint32_t*>(p.o)[static_cast<size_t>(blockIdx.x) * (D / 2) + threadIdx.x] =
            pack_bf16x2(x0, x1);
        if (p.lse != nullptr && threadIdx.x == 0) p.lse[blockIdx.x] = lse_out;
      }
    }
    if (pass == 0) __syncthreads();  // the first pass's sums have been read
  }
}

template <int D, int NQT>
cudaError_t prepare() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void* fn) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               Shape<D, NQT>::kSmem);
  };
  set(reinterpret_cast<const void*>(kv4_decode_split_kernel<D, NQT, Deal::kSplit>));
  set(reinterpret_cast<const void*>(kv4_decode_split_kernel<D, NQT, Deal::kMulti>));
  set(reinterpret_cast<const void*>(kv4_decode_split_kernel<D, NQT, Deal::kDirect>));
  return e;
}

template <int D, int NQT, Deal DEAL>
cudaError_t launch_split(const uint8_t* pool, const Kv4DecodeParams& p, int num_sms,
                         cudaStream_t stream) {
  // kCtasPerSm CTAs per SM, fewer when even the shortest ranges would not fill them
  const int ctas = num_sms * Shape<D, NQT>::kCtasPerSm;
  const int cap = ctas < kKv4MaxRanges / kWarps ? ctas : kKv4MaxRanges / kWarps;
  // a CTA a range first, then more ranges a CTA (the kernel deals them in that order)
  const long long steps = kv4_max_steps(p.S, p.segs, p.max_seq_len);
  const long long want = steps < 1 ? 1 : (steps < num_sms ? steps : num_sms + (steps - num_sms) / kWarps);
  const unsigned grid = DEAL == Deal::kDirect ? static_cast<unsigned>(p.S) * p.segs
                                              : static_cast<unsigned>(want < cap ? want : cap);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Shape<D, NQT>::kSmem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_decode_split_kernel<D, NQT, DEAL>, pool, p);
}

template <int D>
cudaError_t launch(const uint8_t* pool, const Kv4DecodeParams& p, int num_sms, cudaStream_t stream) {
  const bool multi = p.Tq > 1 || p.chunks > 1;
  cudaError_t e;
  if (kv4_direct(p.Tq, p.chunks, p.max_seq_len))
    return p.piece_rows <= 8 ? launch_split<D, 1, Deal::kDirect>(pool, p, num_sms, stream)
                             : launch_split<D, 2, Deal::kDirect>(pool, p, num_sms, stream);
  if (p.piece_rows <= 8)
    e = multi ? launch_split<D, 1, Deal::kMulti>(pool, p, num_sms, stream)
              : launch_split<D, 1, Deal::kSplit>(pool, p, num_sms, stream);
  else
    e = multi ? launch_split<D, 2, Deal::kMulti>(pool, p, num_sms, stream)
              : launch_split<D, 2, Deal::kSplit>(pool, p, num_sms, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.S) * p.Hkv * p.rows);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // Few segments share the ranges among many pieces each: 32 warps a head then (one request
  // of 131000 tokens, 228 pieces a head: 36.6 us a call, 16 warps 37.2, 8 40.6, before the
  // first pass above), else 4, one round trip for the ~15 pieces a head of 64 requests.
  const long long pieces = p.max_pieces / (static_cast<long long>(p.S) * p.segs);
  if (pieces > 48) {
    cfg.blockDim = dim3(32 * 32);
    return cudaLaunchKernelEx(&cfg, kv4_decode_merge_kernel<D, 32>, p);
  }
  cfg.blockDim = dim3(4 * 32);
  return cudaLaunchKernelEx(&cfg, kv4_decode_merge_kernel<D, 4>, p);
}

}  // namespace

long long kv4_max_steps(int S, int segs, int max_seq_len) {
  return static_cast<long long>(S) * segs *
         ((max_seq_len + (kBS * kStepBlocks - 1ll)) / (kBS * kStepBlocks));
}

Kv4Rows kv4_rows(int Hq, int Hkv, int Tq) {
  Kv4Rows r;
  r.rows = Hq / Hkv * Tq;
  r.piece_rows = r.rows < 16 ? r.rows : 16;
  r.chunks = (r.rows + 15) / 16;
  return r;
}

// (a CTA of that form is a whole KV head: rows in several chunks are kMulti's)
bool kv4_direct(int Tq, int chunks, int max_seq_len) {
  return Tq == 1 && chunks == 1 && max_seq_len <= kDirectMaxLen;
}

Kv4DecodeWorkspace kv4_decode_workspace(int S, int Hq, int Hkv, int Tq, int D, int max_seq_len) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  Kv4DecodeWorkspace w{};
  const Kv4Rows r = kv4_rows(Hq, Hkv, Tq);
  if (kv4_direct(Tq, r.chunks, max_seq_len)) return w;
  const long long segs = static_cast<long long>(S) * Hkv * r.chunks;
  const long long steps = kv4_max_steps(S, Hkv * r.chunks, max_seq_len);
  w.pieces = (steps < kKv4MaxRanges ? steps : kKv4MaxRanges) + segs;
  const size_t n = static_cast<size_t>(w.pieces) * r.piece_rows;
  w.off_part_lse = up(n * D * sizeof(float));
  w.off_seg_first = w.off_part_lse + up(n * sizeof(float));
  w.off_seg_last = w.off_seg_first + up(static_cast<size_t>(segs) * sizeof(int));
  w.bytes = w.off_seg_last + up(static_cast<size_t>(segs) * sizeof(int));
  return w;
}

cudaError_t prepare_kv4_decode() {
  cudaError_t e;
  if ((e = prepare<64, 1>()) != cudaSuccess) return e;
  if ((e = prepare<64, 2>()) != cudaSuccess) return e;
  if ((e = prepare<128, 1>()) != cudaSuccess) return e;
  return prepare<128, 2>();
}

cudaError_t launch_kv4_decode(const uint8_t* pool, const Kv4DecodeParams& p, int num_sms,
                              cudaStream_t stream) {
  if (p.S <= 0) return cudaSuccess;
  return p.D == 64 ? launch<64>(pool, p, num_sms, stream) : launch<128>(pool, p, num_sms, stream);
}

}  // namespace gbattn
