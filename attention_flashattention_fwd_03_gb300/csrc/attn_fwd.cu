// attn_fwd.cu -- fused softmax attention forward for sm_103a.
//
// The method (the-ai.news, "Kernels de atencao rapida e fusao de operadores",
// section "Atencao do tipo FlashAttention e atencao paginada"): queries, keys
// and values are processed block by block; for each block a part of the scores
// is computed, the softmax statistics are updated, and the matching output is
// accumulated in on-chip memory, so the Tq x Tk score matrix never reaches HBM.
// The same section describes the paged KV cache (fixed 16-token blocks, every
// logical position translated through a block table); from a paged source the
// key/value tiles are gathered block by block through that table, which is what
// chunked prefill against a paged cache needs.  The paged cache may be held in 4
// bits (kv4.cuh).
//
// GB300 realisation.  One CTA per SM, persistent over work units; a unit is two
// 128-row query tiles of one (batch, head) that share every K/V tile:
//   warp 0        producer: TMA loads of the unit's two Q tiles, then K_j, V_j
//                 into one ring of 128-key slots (128-byte swizzle); in paged
//                 mode lanes 0-7 read the tile's block-table entries (the next
//                 tile's while this one is copied) and each copies its block's
//                 16 rows (of the 4-bit cache: its block's codes and scales, into
//                 a ring of raw half chunks)
//   warp 1        MMA warp (the converged warp runs the issue code; elect.sync
//                 picks the lane that issues): S_i = Q_i K_j^T into TMEM (fp32),
//                 then O_i += P_i V_j with P_i read from TMEM (tcgen05 A operand
//                 in tensor memory), in the order P_0 V_j, S_0(j+1), P_1 V_j,
//                 S_1(j+1); completion is signalled through tcgen05.commit on
//                 mbarriers
//   warps 4-7     softmax of query tile 0, warps 8-11 softmax of tile 1: one
//                 query row per thread (TMEM lane = row).  Each reads S_i from
//                 TMEM, masks, keeps the row max m and sum l, writes
//                 P = 2^(c s - c m) as bf16 back into the S_i columns (c =
//                 scale * log2 e folds the softmax scale into exp2), and at the
//                 end writes O / l (bf16) and LSE = scale m + ln l.
//   warps 12-15   4-bit cache: turn a raw K or V tile into the bf16 slot the MMA
//                 warp reads, 32 keys each.  Every value n s is a bf16 exactly, so
//                 these are the operands themselves, not an approximation of them
//                 (with scales from 2^-123 up, see kv4_values).
//                 On the 16 x 512 workload the 4-bit source takes 435 us where the
//                 bf16 pools take 368 (398 with the four warps passing the slots on
//                 without work: the second hand-over and the ring's missing slot; the
//                 rest are issue slots that the softmax warps lose)
// The two tiles ping-pong: while the softmax warps of one tile work, the tensor
// core computes the other tile's S and P V.  The running max is only moved
// (and O rescaled in TMEM) when a row's max grows by more than 2^8 in exp2
// units, so the rescale is rare; P stays below 2^8, harmless in bf16 and fp32.
// S_i(j+1) completes after P_i(j) V_j (the MMAs of one thread execute in issue
// order), so when the softmax warps see S_i(j+1), O_i is final for tile j and
// the rescale of O_i never waits for the tensor core.
#include <cuda_runtime.h>

#include <cuda_bf16.h>

#include "attn_tile.cuh"
#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

// Where keys and values come from: contiguous tensors, the bf16 pools or the 4-bit pool
// (kSorted..: with the units in order of length, see unit_at).
enum class Src { kContiguous, kPaged, kPaged4, kSortedPaged, kSortedPaged4 };
constexpr bool is_paged(Src s) { return s != Src::kContiguous; }
constexpr bool is_kv4(Src s) { return s == Src::kPaged4 || s == Src::kSortedPaged4; }
constexpr bool is_sorted(Src s) { return s == Src::kSortedPaged || s == Src::kSortedPaged4; }

constexpr int BM = 128;          // query rows per tile (= TMEM lanes)
constexpr int BN = 128;          // keys per K/V tile
constexpr int kBS = 16;          // tokens per paged KV block
// Warpgroup 0: producer, MMA, 2 idle warps; 1, 2: softmax; 3 (4-bit cache): dequantisers.
template <Src SRC>
constexpr int kThreads = is_kv4(SRC) ? 512 : 384;
constexpr float kRescaleLog2 = 8.f;  // move the running max only if it grows by > 2^8
constexpr int kSortLen = 512;    // units are sorted where an item may have more keys than this
constexpr int kMaxSorted = 384;  // (item, query pair) classes whose units are sorted by length
// Registers per thread: the block launches with 168 (384 threads, one block per
// SM); warpgroup 0 gives some up so the softmax warpgroups, which hold a whole
// 128-key score row each, get more: 104 + 200 + 200 = 3 x 168.
constexpr int kRegsLaunch = 168, kRegsWg0 = 104, kRegsSoftmax = 200;
static_assert(kRegsWg0 + 2 * kRegsSoftmax <= 3 * kRegsLaunch, "register split exceeds the launch");
// With the dequantisers the block launches with 128: 80 + 48 + 192 + 192 = 4 x 128 (436 us
// on the 16 x 512 workload; 72 + 56: 440, 88 + 40: 445, 96 + 32: 439).
constexpr int kRegsLaunch4 = 128, kRegsWg0With4 = 80, kRegsDequant = 48, kRegsSoftmax4 = 192;
static_assert(kRegsWg0With4 + kRegsDequant + 2 * kRegsSoftmax4 <= 4 * kRegsLaunch4,
              "register split exceeds the launch");

template <int D, Src SRC>
struct Cfg {
  static constexpr int KB = D / 64;                   // 64-column (128-byte) boxes per row
  static constexpr int BOX_BYTES = 128 * 128;         // 128 rows x 128 bytes
  static constexpr int TILE_BYTES = BM * D * 2;       // one Q, K or V tile
  // K/V ring slots; the raw tiles of the 4-bit cache take the place of one
  static constexpr int NSLOT = (D == 64) ? 8 : (is_kv4(SRC) ? 4 : 5);
  static constexpr int NRAW = is_kv4(SRC) ? 3 : 0;  // raw K or V tiles in flight
  static constexpr int RAW_BLOCK = 9 * D;             // codes and scales of K or V of a block
  static constexpr int RAW_BYTES = (BN / kBS) * RAW_BLOCK;
  static constexpr int OFF_Q = 0;                     // the unit's two Q tiles
  static constexpr int OFF_RING = 2 * TILE_BYTES;
  static constexpr int OFF_RAW = OFF_RING + NSLOT * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_RAW + NRAW * RAW_BYTES;
  static constexpr int NBAR = 2 + 2 * NSLOT + 6 + 1 + 2 * NRAW;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  // sorted units: tile counts and order of the (item, query pair) classes
  static constexpr int OFF_COST = OFF_MISC + 16;
  static constexpr int OFF_ORDER = OFF_COST + (is_sorted(SRC) ? 2 * kMaxSorted : 0);
  static constexpr int OFF_END = OFF_ORDER + (is_sorted(SRC) ? 2 * kMaxSorted : 0);
  static constexpr int SMEM_BYTES = OFF_END + 1024;  // + slack for 1024-byte alignment
  static constexpr uint32_t TMEM_COLS = 512;
  // TMEM columns: S_0 [0,128), S_1 [128,256), O_0 and O_1 from 256 (D each).
  // P_i (bf16 pairs, 64 columns) overwrites the upper half of S_i.
  __device__ static constexpr uint32_t s_col(int i) { return 128u * i; }
  __device__ static constexpr uint32_t p_col(int i) { return 128u * i + 64u; }
  __device__ static constexpr uint32_t o_col(int i) { return 256u + static_cast<uint32_t>(D) * i; }
};
static_assert(kMaxSorted <= kThreads<Src::kSortedPaged>, "a thread a class");
static_assert(Cfg<128, Src::kSortedPaged>::SMEM_BYTES <= 232448, "shared memory budget");
static_assert(Cfg<128, Src::kSortedPaged4>::SMEM_BYTES <= 232448, "shared memory budget");
static_assert(Cfg<64, Src::kSortedPaged4>::SMEM_BYTES <= 232448, "shared memory budget");

template <int D, Src SRC>
struct Bars {
  using C = Cfg<D, SRC>;
  uint32_t base;
  __device__ uint32_t q_full() const { return base; }
  __device__ uint32_t q_empty() const { return base + 8; }
  __device__ uint32_t slot_full(int s) const { return base + 8 * (2 + s); }
  __device__ uint32_t slot_empty(int s) const { return base + 8 * (2 + C::NSLOT + s); }
  __device__ uint32_t s_full(int i) const { return base + 8 * (2 + 2 * C::NSLOT + i); }
  __device__ uint32_t s_free(int i) const { return base + 8 * (4 + 2 * C::NSLOT + i); }
  __device__ uint32_t p_full(int i) const { return base + 8 * (6 + 2 * C::NSLOT + i); }
  __device__ uint32_t teardown() const { return base + 8 * (8 + 2 * C::NSLOT); }
  __device__ uint32_t order() const { return base - C::OFF_BAR + C::OFF_ORDER; }
  __device__ uint32_t raw_full(int s) const { return base + 8 * (9 + 2 * C::NSLOT + s); }
  __device__ uint32_t raw_empty(int s) const { return base + 8 * (9 + 2 * C::NSLOT + C::NRAW + s); }
};

// One work unit: query rows [256 qp, 256 qp + 256) of one (batch, head).
struct Unit {
  int b, bh, kvh, bkv, qp;
  int L;     // keys of this batch item
  int n[2];  // K/V tiles query tile i visits (0: tile past Tq, or no visible key)
  int nkv;   // tiles loaded for the unit = max(n[0], n[1])
  bool bad;  // paged: the batch item's key count is outside its bounds
};

// Keys visible to query row qpos: [0, kv_end).  Causal masks align the last
// query with the last key (query i sits at logical position L - Tq + i).
__device__ __forceinline__ int kv_end_of(int qpos, int L, const FwdParams& p) {
  if (!p.causal) return L;
  const int e = qpos + 1 + (L - p.Tq);
  return e < 0 ? 0 : (e > L ? L : e);
}

// Keys of batch item b, and whether its key count is outside its bounds (then 0).
__device__ __forceinline__ int keys_of(int b, const FwdParams& p, bool paged, bool& bad) {
  bad = false;
  if (!paged) return p.Tk;
  const int L = p.kv_lens[b];
  bad = L < 0 || L > p.max_kv_len || L > p.max_blocks * kBS;
  return bad ? 0 : L;
}

// K/V tiles that query tile i of pair qp visits in an item of L keys.
__device__ __forceinline__ int tiles_of(int qp, int i, int L, const FwdParams& p) {
  const int r0 = 256 * qp + 128 * i;
  if (r0 >= p.Tq) return 0;
  return (kv_end_of(min(r0 + 127, p.Tq - 1), L, p) + BN - 1) / BN;
}

// Unit u: query-pair index decreasing (the longest causal rows first); within one pair
// index, heads of a batch item are adjacent so heads that share K/V run at the same time.
// Sorted: the list at `order` in shared memory holds the classes (qi, b) by decreasing tile
// count, each with its heads adjacent.
//
// Paged items have lengths of their own.  On 16 items of 1024 .. 8192 keys, 1024 units on
// 152 CTAs, the busiest CTA had 1.61 times the mean work in the order of the items and has
// 1.04 times it sorted: bf16 pools 571 -> 368 us, 4-bit 663 -> 438 us.  A unit then costs
// some 0.5 us more to find, and the sort of 300 classes 4 us, so the sorted kernels are taken
// where there is more than one unit a CTA and a bound on the keys above kSortLen; they leave
// the order as it is where no item has more keys than that.  Us, items' order / sorted (D
// 128, bf16 pools, lengths up to the bound): 300 items x 4 heads x 4 rows: 128 keys: 28.9 /
// 37.3, 512: 51.8 / 51.9, 1024: 88.2 / 73.0, 2048: 153 / 116; 40 x 8 x 64: 128: 12.5 / 14.0,
// 512: 21.4 / 18.4, 2048: 51.3 / 38.1; 100 x 16 x 100: 256: 59.8 / 64.1, 1024: 106 / 107,
// 2048: 196 / 166.  Short items under a loose bound stay the dearer: 300 x 4 x 4 rows on up to
// 100 keys 33.0 us with a bound of 8192, 28.6 with one of 100.  Batches of more classes than
// kMaxSorted keep the items' order: 49 items of 2048 rows on 2048 .. 8192 keys (392 classes)
// run at 1376 TFLOP/s, 47 of them (376) at 1473.
template <Src SRC>
__device__ __forceinline__ Unit unit_at(int u, const FwdParams& p, uint32_t order) {
  Unit U;
  int qi;
  if (is_sorted(SRC) && p.B * p.n_qpairs <= kMaxSorted) {
    const int i = u / p.Hq, h = u - i * p.Hq;
    uint16_t cls;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(cls) : "r"(order + 2 * i));
    qi = cls / p.B;
    U.b = cls - qi * p.B;
    U.bh = U.b * p.Hq + h;
    U.kvh = h / p.group;
  } else {
    const int BH = p.B * p.Hq;
    qi = u / BH;
    U.bh = u - qi * BH;
    U.b = U.bh / p.Hq;
    U.kvh = (U.bh - U.b * p.Hq) / p.group;
  }
  U.qp = p.n_qpairs - 1 - qi;
  U.bkv = U.b * p.Hkv + U.kvh;
  U.L = keys_of(U.b, p, is_paged(SRC), U.bad);
#pragma unroll
  for (int i = 0; i < 2; ++i) U.n[i] = tiles_of(U.qp, i, U.L, p);
  U.nkv = max(U.n[0], U.n[1]);
  return U;
}

// Snake order over rounds of gridDim.x units: each CTA alternates between the
// heavier and the lighter end of a round, which evens out causal work.
__device__ __forceinline__ int unit_of_round(int r) {
  return r * static_cast<int>(gridDim.x) +
         ((r & 1) ? static_cast<int>(gridDim.x - 1 - blockIdx.x) : static_cast<int>(blockIdx.x));
}

// ---------------------------------------------------------------------------
// producer warp: TMA loads
// ---------------------------------------------------------------------------
template <int D, Src SRC>
__device__ void producer_warp(const CUtensorMap* tmQ, const CUtensorMap* tmK,
                              const CUtensorMap* tmV, const FwdParams& p, uint32_t sbase,
                              const Bars<D, SRC>& bar, volatile int* abort) {
  using C = Cfg<D, SRC>;
  constexpr bool PAGED = is_paged(SRC);
  constexpr bool RAW = is_kv4(SRC);
  constexpr int NRING = RAW ? C::NRAW : C::NSLOT;  // the ring this warp fills
  const int lane = threadIdx.x & 31;
  const uint32_t sQ = sbase + C::OFF_Q, sR = sbase + (RAW ? C::OFF_RAW : C::OFF_RING);
  auto full = [&](int s) { return RAW ? bar.raw_full(s) : bar.slot_full(s); };
  auto empty = [&](int s) { return RAW ? bar.raw_empty(s) : bar.slot_empty(s); };
  const unsigned long long lim = p.wait_limit_ns;
  int rc = 0, uc = 0;
  bool ok = true, last_q_issued = false;
  for (int r = 0; ok && r * static_cast<int>(gridDim.x) < p.num_units; ++r) {
    const int u = unit_of_round(r);
    if (u >= p.num_units) continue;
    const Unit U = unit_at<SRC>(u, p, bar.order());
    if (PAGED && U.bad && lane == 0) raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
    if (!mbar_wait_warp(bar.q_empty(), (uc & 1) ^ 1, abort, p.flags, lim)) { ok = false; break; }
    last_q_issued = !(p.withhold_copy && uc == 0);  // test hook: withhold the first Q
    if (lane == 0 && last_q_issued) {
      mbar_arrive_expect_tx(bar.q_full(), 2 * C::TILE_BYTES);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
          tma_load_3d(sQ + i * C::TILE_BYTES + kb * C::BOX_BYTES, tmQ, bar.q_full(), kb * 64,
                      256 * U.qp + 128 * i, U.bh);
    }
    ++uc;
    const int nblk_total = (U.L + kBS - 1) / kBS;
    // paged: lane l < 8 reads the table entry of block l of a K/V tile; the next
    // tile's entries are requested before this tile's copies are issued, so the
    // table read is off the copy warp's path
    auto table_entry = [&](int jj) -> int {
      const int nb = min(BN / kBS, nblk_total - jj * (BN / kBS));
      return lane < nb ? p.block_table[static_cast<size_t>(U.b) * p.max_blocks + jj * (BN / kBS) + lane]
                       : 0;
    };
    int next_phys = (PAGED && U.nkv > 0) ? table_entry(0) : 0;
    for (int j = 0; j < U.nkv && ok; ++j) {
      int row_of_lane = 0, nblk = 0;
      if (PAGED) {
        nblk = min(BN / kBS, nblk_total - j * (BN / kBS));
        int phys = next_phys;
        if (j + 1 < U.nkv) next_phys = table_entry(j + 1);
        if (lane < nblk) {
          if (phys < 0 || phys >= p.num_pool_blocks) {
            raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
            phys = 0;
          }
          row_of_lane = (phys * p.Hkv + U.kvh) * kBS;
        }
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const CUtensorMap* map = kv == 0 ? tmK : tmV;
        const int s = rc % NRING;
        if (!mbar_wait_warp(empty(s), ((rc / NRING) & 1) ^ 1, abort, p.flags, lim)) {
          ok = false;
          break;
        }
        const uint32_t dst = sR + s * (RAW ? C::RAW_BYTES : C::TILE_BYTES);
        if (!PAGED) {
          if (lane == 0) {
            mbar_arrive_expect_tx(full(s), C::TILE_BYTES);
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_3d(dst + kb * C::BOX_BYTES, map, full(s), kb * 64, j * BN, U.bkv);
          }
        } else {
          // lane 0 posts the byte count first; then lanes 0..nblk-1 copy their
          // block: 16 rows, one box per 64-column half, or its raw half chunk
          if (lane == 0) mbar_arrive_expect_tx(full(s), nblk * (RAW ? C::RAW_BLOCK : kBS * D * 2));
          __syncwarp();
          if (lane < nblk) {
            if constexpr (RAW) {
              const uint8_t* src =
                  p.kv4_pool + static_cast<size_t>(row_of_lane / kBS) * Kv4<D>::kChunk;
              bulk_load(dst + lane * C::RAW_BLOCK, src + kv * C::RAW_BLOCK, C::RAW_BLOCK, full(s));
            } else {
#pragma unroll
              for (int kb = 0; kb < C::KB; ++kb)
                tma_load_2d(dst + kb * C::BOX_BYTES + lane * kBS * 128, map, full(s), kb * 64,
                            row_of_lane);
            }
          }
          __syncwarp();
        }
        ++rc;
      }
    }
  }
  if (!ok && lane == 0) {
    // Let the copies still in flight land before the CTA's shared memory goes away.
    const unsigned long long quiet = 500000000ull;
    for (int n = (rc > NRING ? rc - NRING : 0); n < rc; ++n)
      mbar_wait_quiet(full(n % NRING), (n / NRING) & 1, quiet);
    if (uc > 0 && last_q_issued) mbar_wait_quiet(bar.q_full(), (uc - 1) & 1, quiet);
  }
}

// ---------------------------------------------------------------------------
// 4-bit cache: warps 12-15 turn raw K and V tiles into bf16 slots, 32 keys each
// ---------------------------------------------------------------------------

// The tiles hold the cache's values / 64 (one operation a pair less, kv4.cuh): the factor
// goes into the softmax scale for keys and into 1 / l for values, exactly.
template <int D, Src SRC>
__device__ void dequant_warp(const FwdParams& p, uint8_t* smem, const Bars<D, SRC>& bar,
                             volatile int* abort) {
  using C = Cfg<D, SRC>;
  using F = Kv4<D>;
  constexpr int G = F::kGroups;
  const int lane = threadIdx.x & 31;
  const int part = (threadIdx.x >> 5) & 3;  // the warp's 32 keys of every tile
  // A lane takes a quarter t of the codes of key `row` of every 8: 8 channels of each
  // group, one 16-byte chunk of the tile.  Rows r and r + 4 are neighbours among the
  // lanes, so that the 8 lanes that store together meet all eight chunk positions of the
  // swizzle.
  const int row = ((lane >> 2) & 1) * 4 + (lane >> 3), t = lane & 3;
  const int out0 = (part * 32 + row) * 128 + ((t ^ row) << 4);  // even groups
  const int out1 = out0 ^ 64;                                   // odd groups
  const unsigned long long lim = p.wait_limit_ns;
  int rc = 0;
  for (int r = 0; r * static_cast<int>(gridDim.x) < p.num_units; ++r) {
    const int u = unit_of_round(r);
    if (u >= p.num_units) continue;
    const Unit U = unit_at<SRC>(u, p, bar.order());
    for (int j = 0; j < U.nkv; ++j) {
#pragma unroll
      for (int kv = 0; kv < 2; ++kv, ++rc) {
        const int rs = rc % C::NRAW, s = rc % C::NSLOT;
        if (!mbar_wait_warp(bar.raw_full(rs), (rc / C::NRAW) & 1, abort, p.flags, lim)) return;
        if (!mbar_wait_warp(bar.slot_empty(s), ((rc / C::NSLOT) & 1) ^ 1, abort, p.flags, lim))
          return;
        const uint8_t* raw = smem + C::OFF_RAW + rs * C::RAW_BYTES;
        uint8_t* tile = smem + C::OFF_RING + s * C::TILE_BYTES;
        const int valid = U.L - j * BN;  // keys past the cache's end become zeros
        // (small loops: unrolled by two they take 464 us against 436, as the code of the
        // roles shares one instruction cache)
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int key = part * 32 + 8 * i + row;
          const uint8_t* blk = raw + (key / kBS) * C::RAW_BLOCK;
          const uint8_t* cp = blk + (key % kBS) * F::kCodeRow + t * (4 * G);
          const uint8_t* sp = blk + kBS * F::kCodeRow + (key % kBS) * F::kScaleRow;
          uint32_t w[G], sc[G / 2];
          if constexpr (G == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(cp);
            const uint2 y = *reinterpret_cast<const uint2*>(sp);
            w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
            sc[0] = y.x, sc[1] = y.y;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(cp);
            w[0] = x.x, w[1] = x.y;
            sc[0] = *reinterpret_cast<const uint32_t*>(sp);
          }
          if (key >= valid) {
#pragma unroll
            for (int g = 0; g < G / 2; ++g) sc[g] = 0;
          }
#pragma unroll
          for (int g = 0; g < G; ++g) {
            // a V row holds 4 channels of every group in turn: a word is put together
            // from the two runs of 4 of its group
            const uint32_t word =
                kv == 0 ? w[g] : __byte_perm(w[g / 2], w[G / 2 + g / 2], (g & 1) ? 0x7632 : 0x5410);
            uint8_t* out = tile + ((g & 1) ? out1 : out0) + (g / 2) * C::BOX_BYTES + i * 1024;
            *reinterpret_cast<uint4*>(out) =
                kv4_values<1>(word, __byte_perm(sc[g / 2], 0, (g & 1) ? 0x3232 : 0x1010));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar.slot_full(s));
          mbar_arrive(bar.raw_empty(rs));
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// MMA warp: the whole warp runs this code, waits together and issues every
// tcgen05.mma and commit from the one lane elect.sync picks (in paged mode it
// also clears key rows past the sequence end in the last V tile).  Shared-memory
// descriptors are built once; an MMA only adds constant offsets to them.
// ---------------------------------------------------------------------------
template <int D, Src SRC>
struct MmaWarp {
  using C = Cfg<D, SRC>;
  static constexpr bool PAGED = is_paged(SRC);
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, 0, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, 0, 1);  // A (P) in TMEM, V MN-major
  static constexpr uint64_t kTileStep = C::TILE_BYTES >> 4;  // descriptor address units

  const FwdParams& p;
  const Bars<D, SRC>& bar;
  volatile int* abort;
  uint32_t sR, tmem;
  uint64_t dq, dk, dv;   // descriptors of Q tile 0 and of ring slot 0 read as K and as V
  int lane;
  int base = 0;          // ring index of the unit's K_0
  int n_pv[2] = {0, 0};  // P V products issued per query tile, all units
  int s_left = 0;        // S products of the unit not yet issued
  int zeroed_j = -1;     // paged: the unit's last V tile has had its dead rows cleared

  __device__ MmaWarp(const FwdParams& p_, const Bars<D, SRC>& b_, volatile int* a_,
                     uint32_t sbase, uint32_t tmem_)
      : p(p_), bar(b_), abort(a_), sR(sbase + C::OFF_RING), tmem(tmem_),
        dq(smem_desc_sw128(sbase + C::OFF_Q, 16, 1024)),
        dk(smem_desc_sw128(sbase + C::OFF_RING, 16, 1024)),
        dv(smem_desc_sw128(sbase + C::OFF_RING, C::BOX_BYTES, 1024)),
        lane(threadIdx.x & 31) {}

  __device__ bool wait(uint32_t b, uint32_t parity) {
    return mbar_wait_warp(b, parity, abort, p.flags, p.wait_limit_ns);
  }
  __device__ int slot(int idx) const { return (base + idx) % C::NSLOT; }
  __device__ uint32_t par(int idx) const { return ((base + idx) / C::NSLOT) & 1; }

  // S_I = Q_I K_j^T.  It overwrites the TMEM columns that P_I of the previous
  // tile occupies; the P V product reading them was issued earlier by this same
  // thread, and one thread's tcgen05.mma operations execute in issue order, so
  // that product has read P_I before this one writes there.
  // Tile 1 uses the ring entries tile 0 has already waited for, whenever tile 0
  // visits the same K/V tile (j < n0); then the phase is known to be complete.
  template <int I>
  __device__ bool issue_s(int j, bool ring_seen) {
    const int ks = slot(2 * j);
    if (!ring_seen && !wait(bar.slot_full(ks), par(2 * j))) return false;
    tc_fence_after();
    const uint64_t a = dq + I * kTileStep, b = dk + static_cast<uint64_t>(ks) * kTileStep;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
      mma_ss_warp(tmem + C::s_col(I), a + off, b + off, kIdescQK, kk > 0 ? 1u : 0u);
    }
    mma_commit_warp(bar.s_full(I));
    if (s_left == 1) mma_commit_warp(bar.q_empty());  // the unit's last read of Q
    --s_left;
    return true;
  }

  // O_I += P_I V_j (P_I from TMEM)
  template <int I>
  __device__ bool issue_pv(int j, int nkv, int L, bool ring_seen) {
    const int vs = slot(2 * j + 1);
    if (!ring_seen && !wait(bar.slot_full(vs), par(2 * j + 1))) return false;
    if (is_paged(SRC) && !is_kv4(SRC) && j == nkv - 1 && zeroed_j != j) {
      zeroed_j = j;
      // Key rows past the sequence end hold stale or arbitrary data (even NaN);
      // their probabilities are 0, but 0 * NaN would reach O.  Clear those rows.
      const int row0 = max(0, L - j * BN);
      uint8_t* gv = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(sR + vs * C::TILE_BYTES));
      for (int e = row0 * 8 + lane; e < BN * 8; e += 32) {  // 8 x 16 bytes per 128-byte row
#pragma unroll
        for (int kb = 0; kb < C::KB; ++kb)
          *reinterpret_cast<uint4*>(gv + kb * C::BOX_BYTES + e * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (!wait(bar.p_full(I), n_pv[I] & 1)) return false;
    tc_fence_after();
    const uint64_t b = dv + static_cast<uint64_t>(vs) * kTileStep;
#pragma unroll
    for (int kk = 0; kk < BN / 16; ++kk)
      mma_ts_warp(tmem + C::o_col(I), tmem + C::p_col(I) + 8 * kk, b + ((kk * 16 * 128) >> 4),
                  kIdescPV, (j > 0 || kk > 0) ? 1u : 0u);
    mma_commit_warp(bar.s_free(I));
    ++n_pv[I];
    return true;
  }

  __device__ void run() {
    int uc = 0;
    for (int r = 0; r * static_cast<int>(gridDim.x) < p.num_units; ++r) {
      const int u = unit_of_round(r);
      if (u >= p.num_units) continue;
      const Unit U = unit_at<SRC>(u, p, bar.order());
      if (!wait(bar.q_full(), uc & 1)) return;
      ++uc;
      const int n0 = U.n[0], n1 = U.n[1], nkv = U.nkv;
      s_left = n0 + n1;
      zeroed_j = -1;
      if (s_left == 0) mma_commit_warp(bar.q_empty());
      if (n0 > 0 && !issue_s<0>(0, false)) return;
      if (n1 > 0 && !issue_s<1>(0, n0 > 0)) return;
      if (nkv > 0) mma_commit_warp(bar.slot_empty(slot(0)));
      for (int j = 0; j < nkv; ++j) {
        if (j < n0 && !issue_pv<0>(j, nkv, U.L, false)) return;
        if (j + 1 < n0 && !issue_s<0>(j + 1, false)) return;
        if (j < n1 && !issue_pv<1>(j, nkv, U.L, j < n0)) return;
        mma_commit_warp(bar.slot_empty(slot(2 * j + 1)));
        if (j + 1 < n1 && !issue_s<1>(j + 1, j + 1 < n0)) return;
        if (j + 1 < nkv) mma_commit_warp(bar.slot_empty(slot(2 * j + 2)));
      }
      base += 2 * nkv;
    }
  }
};

// ---------------------------------------------------------------------------
// softmax warpgroup of query tile I (128 threads, one query row each); both
// warpgroups run this one copy of the code, which keeps the instruction cache
// footprint of the two warpgroups shared
// ---------------------------------------------------------------------------
template <int D, Src SRC>
__device__ void softmax_wg(const FwdParams& p, uint32_t tmem, const Bars<D, SRC>& bar,
                           volatile int* abort, const int I) {
  using C = Cfg<D, SRC>;
  constexpr bool PAGED = is_paged(SRC);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sp = warp & 3;  // TMEM sub-partition this warp may access
  const int r = sp * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
  // (the 4-bit cache's keys come divided by 64)
  const float sl2 = p.scale_log2 * (is_kv4(SRC) ? 64.f : 1.f);
  const float scale = p.scale * (is_kv4(SRC) ? 64.f : 1.f);
  const unsigned long long lim = p.wait_limit_ns;
  int sc = 0;  // S tiles consumed (= P tiles produced), all units

  for (int rr = 0; rr * static_cast<int>(gridDim.x) < p.num_units; ++rr) {
    const int u = unit_of_round(rr);
    if (u >= p.num_units) continue;
    const Unit U = unit_at<SRC>(u, p, bar.order());
    const int n = I ? U.n[1] : U.n[0];
    const int qpos = 256 * U.qp + 128 * I + r;
    const bool row_valid = qpos < p.Tq;
    const int kv_end = row_valid ? kv_end_of(qpos, U.L, p) : U.L;
    float m = -INFINITY, l = 0.f;

    for (int j = 0; j < n; ++j) {
      if (!mbar_wait_warp(bar.s_full(I), sc & 1, abort, p.flags, lim)) return;
      tc_fence_after();
      float s[128];
      {
        uint32_t u32[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(lane_base + C::s_col(I) + 32 * c, u32[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(u32[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int e = 0; e < 32; ++e) s[32 * c + e] = __uint_as_float(u32[c][e]);
      }
      const int kv_lim = kv_end - j * BN;  // keys of this tile visible to the row
      const bool masked = __any_sync(0xffffffffu, kv_lim < BN);
      if (masked) {
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c >= kv_lim) s[c] = -INFINITY;
      }
      const float m_tile = row_max(s);
      // Move the running max only when it grows by more than 2^kRescaleLog2.
      const bool grow = (m_tile - m) * sl2 > kRescaleLog2;
      float alpha = 1.f;
      if (grow) {
        alpha = ex2((m - m_tile) * sl2);  // 0 for the first visible tile (m = -inf)
        m = m_tile;
        l *= alpha;
      }
      if (j > 0 && __any_sync(0xffffffffu, grow)) {
        // O_i already holds P_0..P_{j-1} V (S_i(j) was issued after that product
        // completed): rescale it in TMEM.
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[16];
          tmem_ld16(lane_base + C::o_col(I) + 16 * c, o);
          tmem_wait_ld();
          reg_fence16(o);
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st16(lane_base + C::o_col(I) + 16 * c, o);
        }
        tmem_wait_st();
      }
      const float ms = (m == -INFINITY) ? 0.f : m * sl2;
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      if (masked) {
        write_p<false>(s, sl2, ms, lane_base + C::p_col(I), sum);
      } else {
        write_p<true>(s, sl2, ms, lane_base + C::p_col(I), sum);
      }
      l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar.p_full(I));
      ++sc;
    }

    // epilogue: wait for the last P V, then O / l -> bf16 and LSE
    uint16_t* orow = static_cast<uint16_t*>(p.o) + (static_cast<size_t>(U.bh) * p.Tq + qpos) * D;
    const float nan = __int_as_float(0x7fc00000);
    // no visible key (or none processed); a NaN from the 4-bit cache is a result
    const bool empty = is_kv4(SRC) ? l == 0.f : !(l > 0.f);
    // (the 4-bit cache's values come divided by 64)
    const float inv_l = empty ? 0.f : (is_kv4(SRC) ? 64.f : 1.f) / l;
    if (n > 0) {
      if (!mbar_wait_warp(bar.s_free(I), (sc - 1) & 1, abort, p.flags, lim)) return;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(lane_base + C::o_col(I) + 32 * c, o);
        tmem_wait_ld();
        reg_fence32(o);
        if (row_valid) {
          uint4* dst = reinterpret_cast<uint4*>(orow + 32 * c);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(o[8 * v + e]) * inv_l;
            if (U.bad) {
#pragma unroll
              for (int e = 0; e < 8; ++e) f[e] = nan;
            }
            dst[v] = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
          }
        }
      }
    } else if (row_valid) {
      const uint32_t w = U.bad ? pack_bf16x2(nan, nan) : 0u;
      uint4* dst = reinterpret_cast<uint4*>(orow);
#pragma unroll
      for (int v = 0; v < D / 8; ++v) dst[v] = make_uint4(w, w, w, w);
    }
    if (p.lse != nullptr && row_valid)
      p.lse[static_cast<size_t>(U.bh) * p.Tq + qpos] =
          U.bad ? nan : (empty ? -INFINITY : m * scale + logf(l));
  }
}

template <int D, Src SRC>
__global__ void __launch_bounds__(kThreads<SRC>, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const FwdParams p) {
  using C = Cfg<D, SRC>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const Bars<D, SRC> bar{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(bar.q_full(), 1);
    mbar_init(bar.q_empty(), 1);
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(bar.slot_full(s), is_kv4(SRC) ? 4 : 1);
      mbar_init(bar.slot_empty(s), 1);
    }
    for (int s = 0; s < C::NRAW; ++s) {
      mbar_init(bar.raw_full(s), 1);
      mbar_init(bar.raw_empty(s), 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.s_full(i), 1);
      mbar_init(bar.s_free(i), 1);
      mbar_init(bar.p_full(i), 128);
    }
    mbar_init(bar.teardown(), 1);
    *abort = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  if constexpr (is_kv4(SRC)) {
    // launched as a programmatic dependent: the preceding kernel's writes (an append's) are
    // complete and visible past this point
    asm volatile("griddepcontrol.wait;" ::: "memory");
  }
  if constexpr (is_sorted(SRC)) {
    // every CTA sorts the classes for itself: a class's place is the number of classes
    // before it, by tiles and then by index
    const int classes = p.B * p.n_qpairs;
    if (classes <= kMaxSorted) {
      uint16_t* cost = reinterpret_cast<uint16_t*>(smem + C::OFF_COST);
      uint16_t* places = reinterpret_cast<uint16_t*>(smem + C::OFF_ORDER);
      const int c = threadIdx.x;
      int mine = 0, L = 0;
      if (c < classes) {
        const int qi = c / p.B, qp = p.n_qpairs - 1 - qi;
        bool bad;
        L = keys_of(c - qi * p.B, p, true, bad);
        mine = min(tiles_of(qp, 0, L, p) + tiles_of(qp, 1, L, p), 65535);
        cost[c] = static_cast<uint16_t>(mine);
      }
      const bool sort = __syncthreads_or(L > kSortLen);
      if (c < classes) {
        int place = sort ? 0 : c;
        for (int i = 0; sort && i < classes; ++i)
          place += cost[i] > mine || (cost[i] == mine && i < c);
        places[place] = static_cast<uint16_t>(c);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_decrease<is_kv4(SRC) ? kRegsWg0With4 : kRegsWg0>();
    if (warp == 0) {
      producer_warp<D, SRC>(&tmQ, &tmK, &tmV, p, sbase, bar, abort);
    } else if (warp == 1) {
      MmaWarp<D, SRC> mma(p, bar, abort, sbase, tmem);
      mma.run();
      // Every MMA this warp issued has finished once the teardown barrier flips.
      mma_commit_warp(bar.teardown());
      if (lane == 0) mbar_wait_quiet(bar.teardown(), 0, 1000000000ull);
      __syncwarp();
    }
  } else if (is_kv4(SRC) && warp >= 12) {
    if constexpr (is_kv4(SRC)) {
      regs_decrease<kRegsDequant>();
      dequant_warp<D, SRC>(p, smem, bar, abort);
    }
  } else {
    regs_increase<is_kv4(SRC) ? kRegsSoftmax4 : kRegsSoftmax>();
    softmax_wg<D, SRC>(p, tmem, bar, abort, warp < 8 ? 0 : 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <int D, Src SRC>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(attn_fwd_kernel<D, SRC>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, (Cfg<D, SRC>::SMEM_BYTES));
}

template <int D, Src SRC>
cudaError_t launch(int grid, const CUtensorMap& tmQ, const CUtensorMap& tmK,
                   const CUtensorMap& tmV, const FwdParams& p, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads<SRC>);
  cfg.dynamicSmemBytes = Cfg<D, SRC>::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = is_kv4(SRC) ? 1 : 0;  // the others do not wait for the grid before
  return cudaLaunchKernelEx(&cfg, attn_fwd_kernel<D, SRC>, tmQ, tmK, tmV, p);
}

}  // namespace

cudaError_t prepare_attn_fwd() {
  cudaError_t e;
  if ((e = set_smem<64, Src::kContiguous>()) != cudaSuccess) return e;
  if ((e = set_smem<128, Src::kContiguous>()) != cudaSuccess) return e;
  if ((e = set_smem<64, Src::kPaged>()) != cudaSuccess) return e;
  if ((e = set_smem<128, Src::kPaged>()) != cudaSuccess) return e;
  if ((e = set_smem<64, Src::kPaged4>()) != cudaSuccess) return e;
  if ((e = set_smem<128, Src::kPaged4>()) != cudaSuccess) return e;
  if ((e = set_smem<64, Src::kSortedPaged>()) != cudaSuccess) return e;
  if ((e = set_smem<128, Src::kSortedPaged>()) != cudaSuccess) return e;
  if ((e = set_smem<64, Src::kSortedPaged4>()) != cudaSuccess) return e;
  return set_smem<128, Src::kSortedPaged4>();
}

cudaError_t launch_attn_fwd(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                            const FwdParams& p, int num_sms, cudaStream_t stream) {
  const int grid = p.num_units < num_sms ? p.num_units : num_sms;
  if (grid <= 0) return cudaSuccess;
  auto run = [&](auto d) {
    constexpr int DD = decltype(d)::value;
    const bool sorted = p.num_units > grid && p.max_kv_len > kSortLen;
    if (p.kv4_pool != nullptr)
      return sorted ? launch<DD, Src::kSortedPaged4>(grid, tmQ, tmK, tmV, p, stream)
                    : launch<DD, Src::kPaged4>(grid, tmQ, tmK, tmV, p, stream);
    if (p.block_table != nullptr)
      return sorted ? launch<DD, Src::kSortedPaged>(grid, tmQ, tmK, tmV, p, stream)
                    : launch<DD, Src::kPaged>(grid, tmQ, tmK, tmV, p, stream);
    return launch<DD, Src::kContiguous>(grid, tmQ, tmK, tmV, p, stream);
  };
  return p.D == 64 ? run(std::integral_constant<int, 64>{}) : run(std::integral_constant<int, 128>{});
}

}  // namespace gbattn
