// tree_attn.cu -- attention of the nodes of trees of drafted tokens over the paged cache,
// sm_103a.
//
// A tree's queries share almost all of their keys: the L cached tokens, which every node
// sees, and up to 256 nodes behind them, of which node i sees its ancestors and itself.  So
// the query heads of a KV head and the nodes are rows of one matrix product, every key and
// value is read once for all of them, and only the last tiles of 128 keys need a mask.  A
// row tile holds as many nodes as 128 rows have room for, node by node with the group's heads
// side by side (one TMA box takes them from [Hq, Tn, D]), so that the places past a request's
// last node fill whole tiles, which are not computed.
//
// The work is a sequence of segments, (request, KV head, two row tiles) each, of steps of 128
// keys; a CTA an SM takes an equal range of it, so that one long cache and many short ones
// alike keep every SM busy whatever the lengths.  A segment that is cut between CTAs is put
// together from partial outputs by the merge kernel; whole ones are written at once.  Where
// all caches are short, CTAs take whole segments in turn and there is no merge kernel and no
// workspace.  Trees of more than two row tiles are taken by teams of CTAs, a pair of tiles
// each, over the same keys at the same time, which then come from L2.
//
// A CTA is a pipeline of warps, as in attn_fwd.cu:
//   warp 0      producer: Q tiles, then K and V tiles through the block table (16-row TMA
//               boxes) into a ring
//   warp 1      issues the products: S = Q K^T into tensor memory, O += P V with P from
//               tensor memory
//   warp 2      the segment's tree: its parents, checked
//   warp 3      what there is to do, piece after piece, for all the others (the softmax warps,
//               each thread of which holds a whole score row, have no registers to spare)
//   warps 4-7, 8-11  softmax, a row a thread, of two chains of tiles that alternate on the
//               tensor cores
// With one row tile the two chains take every other key tile, each with its own maximum, sum
// and output, and are joined when the piece ends; with two they take a row tile each over the
// same keys.
//
// What bounds it.  A step is 64 KB (D 128) and, at the copy rate, 1.5 us of an SM's share of HBM;
// with one row tile its products and softmax take 0.5 us, so that HBM bounds it: 64 requests of
// 512 to 8192 tokens x 8 nodes, 12/2 heads (286 MB) take 56.5 us, 75 % of the copy rate, of
// which some 50 stream; one of 131000 tokens x 32 nodes, 32/8 heads (537 MB) 95.5 us, 83 %.  With two
// row tiles a step takes 1.7 us, the pace of attn_fwd.cu (softmax chain and the issue of the
// products): 8 requests x 200 nodes, 32/4 heads (252 GFLOP) 219 us.  What comes on top: some 5 us
// until the first tile is there (plan, table entry, copy, each a round trip, and code that
// is run for the first time), 2 for the last tile and its output, 3 to 10 for the merge.
//
// The probabilities are rounded to bf16 before they multiply V, as in attn_fwd.cu; everything
// else, partial outputs among it, is fp32.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>

#include "api.h"
#include "attn_tile.cuh"
#include "gbattn.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "tree.h"

namespace gbattn {

namespace {

constexpr int BM = 128;  // query rows of a tile
constexpr int BN = 128;  // keys of a step
constexpr int kBS = kPagedBlock;
constexpr int kThreads = 384;
constexpr int kMaxNodes = GBATTN_TREE_MAX_NODES;
constexpr float kRescaleLog2 = 8.f;  // move the running max only if it grows by > 2^8
constexpr int kMaxTeam = 8;
// (each role walking by itself: 61.9 us instead of 58.3 on 64 requests x 8 nodes)
constexpr int kPieces = 4;           // pieces told ahead
constexpr int kRoles = 11;           // warps that are told
// Registers of the first four warps and of the softmax warps: the block launches with 168 a thread,
// and neither side spills.  (104 + 200 for both forms: 200 nodes 220 us instead of 217.6.)
constexpr int kRegsLaunch = 168;
constexpr int regs_wg0(bool split) { return split ? 88 : 120; }
constexpr int regs_softmax(bool split) { return split ? 208 : 192; }
static_assert(regs_wg0(true) + 2 * regs_softmax(true) <= 3 * kRegsLaunch &&
                  regs_wg0(false) + 2 * regs_softmax(false) <= 3 * kRegsLaunch,
              "register split exceeds the launch");
constexpr float kNan = __builtin_nanf("");

// The steps lie on a line: a segment begins with kSegCost (queries to be fetched, an output to be
// written), then its steps follow one another at the distance of what one costs.  A range takes
// the steps that lie in it.  With kSegCost 10 / 20 / 32, 64 requests x 8 nodes take 58.1 / 57.6 /
// 58.7 us, 16 x up to 64 nodes 69.3 / 66.4 / 66.8; with kStepCost2 24 the latter 71.3.
constexpr int kSegCost = 20;
constexpr int kStepCost0 = 4, kStepCost1 = 16, kStepCost2 = 20;  // by row tiles (0: zeros are written)
constexpr int kMostCost = kSegCost + kStepCost2;  // no range is shorter, so that each holds a step

struct Plan {        // this CTA's range
  int lo, hi;        // where it begins and ends
  int pos, r, s, j;  // the first step's place, request, segment of the request and step of that
  int share, extra;
};

// The rows of a CTA that are cut after its range and begin in it: request, KV head, pair of row
// tiles and how many of the two there are, number of pieces and the first one's slot (the others
// are the first slots of the CTAs that go on).
struct Cut {
  int r, kvh, pair, tiles, pieces, slot;
};

struct Work {  // what the kernels share besides the caller's operands
  TreeParams p;
  float* part_o;    // [2 grid][D / 4][unit_rows][4]: a warp's rows side by side
  float* part_lse;  // [2 grid][unit_rows]
  Cut* cut;         // [grid]
  int group;        // query heads of a KV head
  int per_group;    // 2^16 / group, rounded up: x per_group >> 16 = x / group for x < 128
  int tile_nodes;   // nodes of a row tile
  int pairs;        // pairs of row tiles of a KV head
  int team;         // CTAs of a team: pairs that are taken together
  int rounds;       // teams' turns at a KV head
  int segs;         // Hkv * rounds
  int unit_rows;    // rows of a partial output
  int direct;       // teams take whole segments in turn
};

// The part of a segment that a CTA takes.
struct Piece {
  int r, kvh, pair;
  int L, nodes;   // of the request: tokens before the tree, nodes of it
  int j0, n;      // first key tile and how many (0: nothing to compute; -1: no more pieces)
  int row_tiles;  // of the pair's two, how many hold nodes
  int slot;       // of its partial output; -1: the segment is whole
  int last;       // holds the segment's last step
  int bad;        // the request's sizes are out of bounds
  int tail;       // some of its tiles hold nodes' keys
};

// A checked tree: the parent of each node + 1, and the first node of the chain of consecutive
// numbers that ends with it.
template <int N>
struct Tree {
  uint8_t parent1[N], start[N];
};

template <int D, bool SPLIT>
struct Cfg {
  static constexpr int KB = D / 64;              // 64-column (128-byte) boxes of a row
  static constexpr int BOX_BYTES = BM * 128;
  static constexpr int TILE_BYTES = BM * D * 2;
  static constexpr int NQ = SPLIT ? 1 : 2;       // row tiles
  // (D 128, one row tile: 5 slots 57.8 us on 64 requests x 8 nodes, 97.2 on 131000 tokens; 6 slots
  // 57.4 and 96.4; 4 slots 2 and 4 us more than 5)
  static constexpr int NSLOT = D == 64 ? 8 : (SPLIT ? 6 : 5);
  using Nodes = Tree<SPLIT ? BM : kMaxNodes>;    // (in one row tile: 128 at most)
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = NQ * TILE_BYTES;
  static constexpr int OFF_TREE = OFF_RING + NSLOT * TILE_BYTES;  // [2] Tree
  static constexpr int OFF_JOIN = OFF_TREE + 2 * sizeof(Nodes);   // SPLIT: [2][BM] float2, maximum and sum
  static constexpr int OFF_BAR = OFF_JOIN + (SPLIT ? 2 * BM * 8 : 0);
  static constexpr int NBAR = 2 + 2 * NSLOT + 6 + 1 + 4 + 2 + 2 * kPieces;
  static constexpr int OFF_PIECES = OFF_BAR + NBAR * 8;                   // [kPieces]
  static constexpr int OFF_MISC = OFF_PIECES + kPieces * sizeof(Piece);   // TMEM address, abort, bad tree [2]
  // the plan, and sums [12] for it, are over before the first join
  static constexpr int OFF_PLAN = SPLIT ? OFF_JOIN : OFF_MISC + 16;
  static constexpr int OFF_SUMS = OFF_PLAN + sizeof(Plan);
  static constexpr int END = SPLIT ? OFF_MISC + 16 : OFF_SUMS + 48;
  // Room to align to 1024 bytes by hand, unless there is none: the array is declared with that
  // alignment, and the kernel checks it.
  static constexpr int SLACK = END + 1024 <= 232448 ? 1024 : 0;
  static constexpr int SMEM_BYTES = END + SLACK;
  static constexpr uint32_t TMEM_COLS = 512;
  // TMEM columns: S_0 [0,128), S_1 [128,256), O_0 and O_1 from 256 (D each).  P_i (bf16
  // pairs, 64 columns) overwrites the upper half of S_i.
  __device__ static constexpr uint32_t s_col(int i) { return 128u * i; }
  __device__ static constexpr uint32_t p_col(int i) { return 128u * i + 64u; }
  __device__ static constexpr uint32_t o_col(int i) { return 256u + static_cast<uint32_t>(D) * i; }
};
static_assert(Cfg<128, true>::SMEM_BYTES <= 232448 && Cfg<128, false>::SMEM_BYTES <= 232448,
              "shared memory budget");

template <int D, bool SPLIT>
struct Bars {
  using C = Cfg<D, SPLIT>;
  uint32_t base;
  __device__ uint32_t at(int i) const { return base + 8 * i; }
  __device__ uint32_t q_full() const { return at(0); }
  __device__ uint32_t q_empty() const { return at(1); }
  __device__ uint32_t slot_full(int s) const { return at(2 + s); }
  __device__ uint32_t slot_empty(int s) const { return at(2 + C::NSLOT + s); }
  __device__ uint32_t s_full(int i) const { return at(2 + 2 * C::NSLOT + i); }
  __device__ uint32_t s_free(int i) const { return at(4 + 2 * C::NSLOT + i); }
  __device__ uint32_t p_full(int i) const { return at(6 + 2 * C::NSLOT + i); }
  __device__ uint32_t teardown() const { return at(8 + 2 * C::NSLOT); }
  __device__ uint32_t tree_full(int b) const { return at(9 + 2 * C::NSLOT + b); }
  __device__ uint32_t tree_empty(int b) const { return at(11 + 2 * C::NSLOT + b); }
  __device__ uint32_t joined(int i) const { return at(13 + 2 * C::NSLOT + i); }
  __device__ uint32_t piece_full(int i) const { return at(15 + 2 * C::NSLOT + i); }
  __device__ uint32_t piece_empty(int i) const { return at(15 + 2 * C::NSLOT + kPieces + i); }
};

// A request's sizes: tokens before the tree, nodes, and whether they are out of bounds (then
// the request counts as empty).
struct Sizes {
  int L, n;
  bool bad;
  // (unsigned: the keys may come to 2^31 - 16)
  __device__ int tiles() const { return static_cast<int>((static_cast<unsigned>(L + n) + (BN - 1)) / BN); }
};
__device__ __forceinline__ Sizes sizes_of(const TreeParams& p, int r) {
  Sizes z{p.seq_lens[r], p.tree_lens ? p.tree_lens[r] : p.Tn, false};
  const long long keys = static_cast<long long>(z.L) + z.n;
  z.bad = z.L < 0 || z.n < 0 || z.n > p.Tn || keys > p.max_seq_len ||
          keys > static_cast<long long>(p.max_blocks) * kBS;
  if (z.bad) z.L = z.n = 0;
  return z;
}
// Row tiles of a request that hold nodes, pairs of them, and team rounds with such a pair.
__device__ __forceinline__ int live_tiles(const Work& w, const Sizes& z) {
  return (z.n + w.tile_nodes - 1) / w.tile_nodes;
}
__device__ __forceinline__ int live_pairs(const Work& w, const Sizes& z) {
  return (live_tiles(w, z) + 1) / 2;
}
__device__ __forceinline__ int live_rounds(const Work& w, const Sizes& z) {
  return (live_pairs(w, z) + w.team - 1) / w.team;
}
// Steps of a segment (without nodes one, in which zeros are written) and what one costs.
__device__ __forceinline__ int steps_of(const Work& w, const Sizes& z, int round) {
  return round < live_rounds(w, z) ? z.tiles() : 1;
}
__device__ __forceinline__ int step_cost(const Work& w, const Sizes& z, int round) {
  const int tiles = live_tiles(w, z) - 2 * round * w.team;
  return tiles <= 0 ? kStepCost0 : (tiles == 1 ? kStepCost1 : kStepCost2);
}

// Walks over this CTA's pieces.
struct Walk {
  const Work& w;
  int team, member;
  int at;  // place of the next step on the line, or (direct) the next segment
  int hi, r, s, j, index = 0;
  int end = 0;  // where the segment of the last piece ends on the line (not if direct)
  Sizes z;
  __device__ Walk(const Work& w_, const Plan& plan)
      : w(w_), team(blockIdx.x / w_.team), member(blockIdx.x - team * w_.team),
        at(w_.direct ? team : plan.pos), hi(w_.direct ? w_.p.S * w_.segs : plan.hi),
        r(w_.direct ? -1 : plan.r), s(plan.s), j(plan.j) {
    if (!w.direct && at < hi) z = sizes_of(w.p, r);
  }
  __device__ bool next(Piece& x) {
    if (at >= hi) return false;
    if (w.direct) {
      const int now = at / w.segs;
      if (now != r) z = sizes_of(w.p, now);
      r = now;
      s = at - now * w.segs;
      at += gridDim.x / w.team;
      j = 0;
    }
    x.kvh = s / w.rounds;
    const int round = s - x.kvh * w.rounds;
    const int steps = steps_of(w, z, round), cost = step_cost(w, z, round);
    if (j >= steps) {  // (lengths changed under the kernel)
      at = hi;
      return false;
    }
    const int n = w.direct ? steps : min((hi - at + cost - 1) / cost, steps - j);
    const int tiles = live_tiles(w, z);
    x.r = r;
    x.pair = round * w.team + member;
    x.L = z.L;
    x.nodes = z.n;
    x.row_tiles = max(0, min(2, tiles - 2 * x.pair));
    x.j0 = j;
    x.n = x.row_tiles > 0 ? n : 0;
    x.last = j + n == steps;
    x.bad = z.bad;
    x.tail = x.n > 0 && z.L - (j + n - 1) * BN < BN;
    x.slot = j == 0 && x.last ? -1 : 2 * static_cast<int>(blockIdx.x) + (index > 0 ? 1 : 0);
    ++index;
    if (!w.direct) {
      end = at + (steps - j) * cost;
      at += n * cost;
      j += n;
      if (j == steps) {
        at += kSegCost;
        j = 0;
        if (at < hi && ++s == w.segs) {
          s = 0;
          if (++r >= w.p.S) at = hi;  // (lengths changed under the kernel)
          else z = sizes_of(w.p, r);
        }
      }
    }
    return true;
  }
};

// ---------------------------------------------------------------------------
// warp 3: tells the other roles what to do
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
__device__ void planner_warp(const Work& w, const Plan plan, uint8_t* smem, const Bars<D, SPLIT>& bar,
                             volatile int* abort) {  // (one lane)
  using C = Cfg<D, SPLIT>;
  const TreeParams& p = w.p;
  Piece* pieces = reinterpret_cast<Piece*>(smem + C::OFF_PIECES);
  Cut cut{0, 0, 0, 0, 0, 0};
  Walk walk(w, plan);
  Piece x;
  for (int i = 0;; ++i) {
    const bool more = walk.next(x);
    if (!more) x.n = -1;
    if (!mbar_wait(bar.piece_empty(i % kPieces), ((i / kPieces) & 1) ^ 1, abort, p.flags, p.wait_limit_ns)) {
      cut.pieces = 0;  // (what there is need not have been computed)
      break;
    }
    pieces[i % kPieces] = x;
    mbar_arrive(bar.piece_full(i % kPieces));
    if (!more) break;
    if (x.bad) raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
    if (!w.direct && !x.last && x.j0 == 0 && x.n > 0) {  // (the range's last piece, then)
      // the rows go on up to the range that holds the segment's last step
      const int e = walk.end - step_cost(w, walk.z, x.pair / w.team), big = plan.extra * (plan.share + 1);
      const int k1 = e < big ? e / (plan.share + 1) : plan.extra + (e - big) / plan.share;
      // (within the launch, should the lengths have changed under the kernel)
      const int pieces = min(k1, static_cast<int>(gridDim.x) / w.team - 1) - walk.team + 1;
      cut = Cut{x.r, x.kvh, x.pair, x.row_tiles, pieces, x.slot};
    }
  }
  if (!w.direct) w.cut[blockIdx.x] = cut;
}

// A field of a piece, by the piece's shared-memory address; the whole warp calls this together.
// All lanes read the same: the shuffle
// tells the compiler so, which then keeps loops over it and what the products are issued with in
// uniform registers (8 requests x 200 nodes: 234 us, 242 with plain reads).
__device__ __forceinline__ int field_at(uint32_t x, uint32_t offset) {
  int v;
  asm volatile("ld.shared.s32 %0, [%1];" : "=r"(v) : "r"(x + offset) : "memory");
  return __shfl_sync(0xffffffffu, v, 0);
}
#define FIELD(x, name) field_at(x, offsetof(Piece, name))

// A warp's view of the pieces.
template <int D, bool SPLIT>
struct Feed {
  using C = Cfg<D, SPLIT>;
  const Bars<D, SPLIT>& bar;
  int i = 0;
  __device__ explicit Feed(const Bars<D, SPLIT>& b) : bar(b) {}
  // The next piece's address, or 0 (after the last one, or the CTA is stopping).
  __device__ uint32_t next(const TreeParams& p, volatile int* abort) {
    if (!mbar_wait_warp(bar.piece_full(i % kPieces), (i / kPieces) & 1, abort, p.flags, p.wait_limit_ns))
      return 0;
    const uint32_t x = bar.base - C::OFF_BAR + C::OFF_PIECES + (i % kPieces) * sizeof(Piece);
    return FIELD(x, n) < 0 ? 0 : x;
  }
  __device__ void done() {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar.piece_empty(i % kPieces));
    ++i;
  }
};

// ---------------------------------------------------------------------------
// producer warp
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
__device__ void producer_warp(const CUtensorMap* tmQ, const CUtensorMap* tmK,
                              const CUtensorMap* tmV, const Work& w,
                              uint32_t sbase, const Bars<D, SPLIT>& bar, volatile int* abort) {
  using C = Cfg<D, SPLIT>;
  const TreeParams& p = w.p;
  const int lane = threadIdx.x & 31;
  const uint32_t sQ = sbase + C::OFF_Q, sR = sbase + C::OFF_RING;
  const unsigned long long lim = p.wait_limit_ns;
  const uint64_t stream_policy = l2_policy_evict_first();
  // every K/V byte is read once, and may go first (58.0 us; kept like the rest 59.6)
  const bool once = w.team == 1 && w.rounds == 1;
  int rc = 0, uc = 0;
  bool ok = true, last_q_issued = false;
  Feed<D, SPLIT> feed(bar);
  for (uint32_t x; ok && (x = feed.next(p, abort)); feed.done()) {
    const int n = FIELD(x, n), r = FIELD(x, r), kvh = FIELD(x, kvh), j0 = FIELD(x, j0), j1 = j0 + n;
    if (n == 0) continue;
    const int row_tiles = FIELD(x, row_tiles), node0 = 2 * FIELD(x, pair) * w.tile_nodes;
    const int blocks = (FIELD(x, L) + FIELD(x, nodes) + kBS - 1) / kBS;
    // lane l < 8 reads the table entry of block l of a tile, one tile ahead of the copies
    auto table_entry = [&](int j) -> int {
      const int b = j * (BN / kBS) + lane;
      return lane < BN / kBS && b < blocks
                 ? p.block_table[static_cast<size_t>(r) * p.max_blocks + b]
                 : 0;
    };
    int next_phys = table_entry(j0);
    for (int j = j0; j < j1 && ok; ++j) {
      const int nblk = min(BN / kBS, blocks - j * (BN / kBS));
      int phys = next_phys, row = 0;
      if (j + 1 < j1) next_phys = table_entry(j + 1);
      if (lane < nblk) {
        if (phys < 0 || phys >= p.num_pool_blocks) {
          raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
          phys = 0;
        }
        row = (phys * p.Hkv + kvh) * kBS;
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const CUtensorMap* map = kv == 0 ? tmK : tmV;
        const int s = rc % C::NSLOT;
        if (!mbar_wait_warp(bar.slot_empty(s), ((rc / C::NSLOT) & 1) ^ 1, abort, p.flags, lim)) {
          ok = false;
          break;
        }
        const uint32_t dst = sR + s * C::TILE_BYTES;
        // lane 0 posts the byte count first
        if (lane == 0) mbar_arrive_expect_tx(bar.slot_full(s), nblk * kBS * D * 2);
        __syncwarp();
        if (lane < nblk) {
#pragma unroll
          for (int kb = 0; kb < C::KB; ++kb) {
            if (once)
              tma_load_2d_hint(dst + kb * C::BOX_BYTES + lane * kBS * 128, map, bar.slot_full(s),
                               kb * 64, row, stream_policy);
            else
              tma_load_2d(dst + kb * C::BOX_BYTES + lane * kBS * 128, map, bar.slot_full(s),
                          kb * 64, row);
          }
        }
        __syncwarp();
        ++rc;
      }
      if (ok && j == j0) {
        // the queries go behind the first tile, whose slots are free before the piece before is
        // done with its own queries
        if (!mbar_wait_warp(bar.q_empty(), (uc & 1) ^ 1, abort, p.flags, lim)) {
          ok = false;
          break;
        }
        last_q_issued = !(p.withhold_copy && uc == 0);  // test hook: withhold the first Q
        if (lane == 0 && last_q_issued) {
          mbar_arrive_expect_tx(bar.q_full(), row_tiles * C::KB * w.group * w.tile_nodes * 128);
          for (int i = 0; i < row_tiles; ++i)
#pragma unroll
            for (int kb = 0; kb < C::KB; ++kb)
              tma_load_4d(sQ + i * C::TILE_BYTES + kb * C::BOX_BYTES, tmQ, bar.q_full(), kb * 64, 0,
                          node0 + i * w.tile_nodes, r * p.Hkv + kvh);
        }
        ++uc;
      }
    }
  }
  if (!ok && lane == 0) {
    // Let the copies still in flight land before the CTA's shared memory goes away.
    const unsigned long long quiet = 500000000ull;
    for (int n = (rc > C::NSLOT ? rc - C::NSLOT : 0); n < rc; ++n)
      mbar_wait_quiet(bar.slot_full(n % C::NSLOT), (n / C::NSLOT) & 1, quiet);
    if (uc > 0 && last_q_issued) mbar_wait_quiet(bar.q_full(), (uc - 1) & 1, quiet);
  }
}

// ---------------------------------------------------------------------------
// warp 2: the trees
// ---------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ bool read_tree(const int32_t* parents, int n, Tree<N>& tree) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  int before = 0;  // start of the chain that ends with the node before
  for (int b = 0; b < n; b += 32) {
    const int i = b + lane;
    int a = i < n ? parents[i] : -1;
    const bool wrong = a < -1 || a >= i;
    bad |= i < n && wrong;
    if (wrong) a = -1;
    int start = a == i - 1 ? 0 : i;  // the largest break so far
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, start, o);
      if (lane >= o) start = max(start, v);
    }
    start = max(start, before);
    before = __shfl_sync(0xffffffffu, start, 31);
    if (i < n) {
      tree.parent1[i] = static_cast<uint8_t>(a + 1);
      tree.start[i] = static_cast<uint8_t>(start);
    }
  }
  return __any_sync(0xffffffffu, bad);
}

template <int D, bool SPLIT>
__device__ void tree_warp(const Work& w, uint8_t* smem, const Bars<D, SPLIT>& bar,
                          volatile int* abort) {
  using C = Cfg<D, SPLIT>;
  const TreeParams& p = w.p;
  const int lane = threadIdx.x & 31;
  volatile int* bad_tree = reinterpret_cast<volatile int*>(smem + C::OFF_MISC) + 2;
  int mc = 0;
  Feed<D, SPLIT> feed(bar);
  for (uint32_t x; (x = feed.next(p, abort)); feed.done()) {
    if (!FIELD(x, tail)) continue;
    const int b = mc & 1;
    if (!mbar_wait_warp(bar.tree_empty(b), ((mc >> 1) & 1) ^ 1, abort, p.flags, p.wait_limit_ns)) return;
    const bool bad = read_tree(p.parents + static_cast<size_t>(FIELD(x, r)) * p.Tn, FIELD(x, nodes),
                               reinterpret_cast<typename C::Nodes*>(smem + C::OFF_TREE)[b]);
    if (lane == 0) {
      bad_tree[b] = bad;
      if (bad) raise_flag(p.flags, DEVFLAG_BAD_TREE);
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(bar.tree_full(b));
    ++mc;
  }
}

// ---------------------------------------------------------------------------
// MMA warp (the converged warp runs the issue code, elect.sync picks the issuing lane)
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
struct MmaWarp {
  using C = Cfg<D, SPLIT>;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(BM, BN, 0, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(BM, D, 0, 1);  // P in TMEM, V MN-major
  static constexpr uint64_t kTileStep = C::TILE_BYTES >> 4;

  const Work& w;
  const Bars<D, SPLIT>& bar;
  volatile int* abort;
  uint32_t sR, tmem;
  uint64_t dq, dk, dv;  // descriptors of Q tile 0 and of ring slot 0 read as K and as V
  int lane;
  int base = 0;          // ring index of the piece's first K tile
  int n_pv[2] = {0, 0};  // P V products issued per chain, all pieces
  int cleared = -1;      // the piece's last V tile has had its dead rows cleared

  __device__ MmaWarp(const Work& w_, const Bars<D, SPLIT>& b_, volatile int* a_, uint32_t sbase,
                     uint32_t tmem_)
      : w(w_), bar(b_), abort(a_), sR(sbase + C::OFF_RING), tmem(tmem_),
        dq(smem_desc_sw128(sbase + C::OFF_Q, 16, 1024)),
        dk(smem_desc_sw128(sbase + C::OFF_RING, 16, 1024)),
        dv(smem_desc_sw128(sbase + C::OFF_RING, C::BOX_BYTES, 1024)),
        lane(threadIdx.x & 31) {}

  __device__ bool wait(uint32_t b, uint32_t parity) {
    return mbar_wait_warp(b, parity, abort, w.p.flags, w.p.wait_limit_ns);
  }
  __device__ int slot(int i) const { return (base + i) % C::NSLOT; }
  __device__ uint32_t par(int i) const { return ((base + i) / C::NSLOT) & 1; }

  // S_I = Q_I K_t^T (t counts the piece's tiles).  It overwrites the columns of P_I of the
  // tile before, whose P V product was issued earlier by this same thread: one thread's
  // products execute in issue order.
  template <int I>
  __device__ bool issue_s(int t, bool ring_seen) {
    const int ks = slot(2 * t);
    if (!ring_seen && !wait(bar.slot_full(ks), par(2 * t))) return false;
    tc_fence_after();
    const uint64_t a = dq + (SPLIT ? 0 : I) * kTileStep, b = dk + static_cast<uint64_t>(ks) * kTileStep;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const uint32_t off = ((kk >> 2) * C::BOX_BYTES + (kk & 3) * 32) >> 4;
      mma_ss_warp(tmem + C::s_col(I), a + off, b + off, kIdescQK, kk > 0 ? 1u : 0u);
    }
    mma_commit_warp(bar.s_full(I));
    return true;
  }

  // O_I += P_I V_t (P_I from TMEM); `add`: the chain has an earlier tile in this piece
  template <int I>
  __device__ bool issue_pv(int t, bool add, int dead_from, bool ring_seen) {
    const int vs = slot(2 * t + 1);
    if (!ring_seen && !wait(bar.slot_full(vs), par(2 * t + 1))) return false;
    if (dead_from < BN && cleared != t) {
      cleared = t;
      // Rows past the last key hold stale or arbitrary data (even NaN); their probabilities
      // are 0, but 0 * NaN would reach O.
      uint8_t* gv = reinterpret_cast<uint8_t*>(__cvta_shared_to_generic(sR + vs * C::TILE_BYTES));
      for (int e = dead_from * 8 + lane; e < BN * 8; e += 32) {  // 8 x 16 bytes a 128-byte row
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
                  kIdescPV, (add || kk > 0) ? 1u : 0u);
    mma_commit_warp(bar.s_free(I));
    ++n_pv[I];
    return true;
  }

  __device__ void run() {
    int uc = 0;
    Feed<D, SPLIT> feed(bar);
    for (uint32_t x; (x = feed.next(w.p, abort)); feed.done()) {
      const int n = FIELD(x, n);
      if (n == 0) continue;
      if (!wait(bar.q_full(), uc & 1)) return;
      ++uc;
      cleared = -1;
      // row of the last tile from which on there are no keys
      const int keys_left = FIELD(x, L) + FIELD(x, nodes) - FIELD(x, j0) * BN;
      auto dead_from = [&](int t) { return keys_left - t * BN; };
      if (SPLIT) {
        if (!issue_s<0>(0, false)) return;
        mma_commit_warp(bar.slot_empty(slot(0)));
        if (n > 1) {
          if (!issue_s<1>(1, false)) return;
          mma_commit_warp(bar.slot_empty(slot(2)));
        }
        if (n <= 2) mma_commit_warp(bar.q_empty());
        for (int t = 0; t < n; ++t) {
          if (!(t & 1 ? issue_pv<1>(t, t > 1, dead_from(t), false)
                      : issue_pv<0>(t, t > 1, dead_from(t), false)))
            return;
          mma_commit_warp(bar.slot_empty(slot(2 * t + 1)));
          if (t + 2 < n) {
            if (!(t & 1 ? issue_s<1>(t + 2, false) : issue_s<0>(t + 2, false))) return;
            mma_commit_warp(bar.slot_empty(slot(2 * t + 4)));
            if (t + 3 == n) mma_commit_warp(bar.q_empty());  // the piece's last read of Q
          }
        }
      } else {
        const bool two = FIELD(x, row_tiles) == 2;
        if (!issue_s<0>(0, false)) return;
        if (two && !issue_s<1>(0, true)) return;
        mma_commit_warp(bar.slot_empty(slot(0)));
        if (n == 1) mma_commit_warp(bar.q_empty());
        for (int t = 0; t < n; ++t) {
          if (!issue_pv<0>(t, t > 0, dead_from(t), false)) return;
          if (t + 1 < n && !issue_s<0>(t + 1, false)) return;
          if (two && !issue_pv<1>(t, t > 0, dead_from(t), true)) return;
          mma_commit_warp(bar.slot_empty(slot(2 * t + 1)));
          if (t + 1 < n) {
            if (two && !issue_s<1>(t + 1, true)) return;
            mma_commit_warp(bar.slot_empty(slot(2 * t + 2)));
            if (t + 2 == n) mma_commit_warp(bar.q_empty());
          }
        }
      }
      base += 2 * n;
    }
  }
};

// What node a sees of the 32 keys from x on, x counted from node 0 (the keys before it are the
// cached tokens); a becomes the first of its ancestors before those keys.
template <int N>
__device__ __forceinline__ uint32_t seen_bits(const Tree<N>& tree, int& a, int x) {
  uint32_t bits = x <= -32 ? 0xffffffffu : (x < 0 ? (1u << -x) - 1u : 0u);
  while (a >= max(x, 0)) {
    const int s = tree.start[a];  // s .. a are its own or its ancestors
    const int hi = min(a - x, 31), lo = max(s - x, 0);
    if (lo <= hi) bits |= (0xffffffffu >> (31 - hi)) & (0xffffffffu << lo);
    a = s < x ? x - 1 : tree.parent1[s] - 1;
  }
  return bits;
}

// ---------------------------------------------------------------------------
// softmax warpgroup of chain I (128 threads, one query row each)
// ---------------------------------------------------------------------------
template <int D, bool SPLIT>
__device__ void softmax_wg(const Work& w, uint8_t* smem, uint32_t tmem,
                           const Bars<D, SPLIT>& bar, volatile int* abort, const int I) {
  using C = Cfg<D, SPLIT>;
  const TreeParams& p = w.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sp = warp & 3;  // TMEM sub-partition this warp may access
  const int tile_row = sp * 32 + lane;
  const uint32_t lane_base = tmem + (static_cast<uint32_t>(sp * 32) << 16);
  const float sl2 = p.scale_log2;
  const unsigned long long lim = p.wait_limit_ns;
  volatile int* bad_trees = reinterpret_cast<volatile int*>(smem + C::OFF_MISC) + 2;
  float2* join = reinterpret_cast<float2*>(smem + C::OFF_JOIN);
  int sc = 0;  // tiles consumed by this chain, all pieces
  int mc = 0;  // masks consumed
  int jc = 0;  // pieces joined
  // A meeting of both warpgroups, with a bounded wait like every other.
  auto meet = [&](int i) {
    tc_fence_before();
    mbar_arrive(bar.joined(i));
    if (!mbar_wait_warp(bar.joined(i), jc & 1, abort, p.flags, lim)) return false;
    tc_fence_after();
    return true;
  };
  // node of the row tile and head of this thread's row
  auto place = [&]() {
    // (rows behind the tile's nodes get a head that does not exist)
    const int node = (tile_row * w.per_group) >> 16, head = tile_row - node * w.group;
    return node < w.tile_nodes ? node | head << 8 : 255 | 255 << 8;
  };
  const auto* trees = reinterpret_cast<const typename C::Nodes*>(smem + C::OFF_TREE);
  Feed<D, SPLIT> feed(bar);
  for (uint32_t x; (x = feed.next(p, abort)); feed.done()) {
    const int total = FIELD(x, n), L = FIELD(x, L);
    int j = FIELD(x, j0) + (SPLIT ? I : 0);
    const int n = SPLIT ? (total + 1 - I) / 2 : (I < FIELD(x, row_tiles) ? total : 0);
    // this row's node (-1: none is in this place); a warp without any only keeps step
    const int nodes = FIELD(x, nodes), pair = FIELD(x, pair);
    int node = (2 * pair + (SPLIT ? 0 : I)) * w.tile_nodes + (place() & 255);
    if (node >= nodes) node = -1;
    const bool live = __any_sync(0xffffffffu, node >= 0);
    const int b = mc & 1;
    bool have_mask = false;
    float m = -INFINITY, l = 0.f;
    for (int i = 0; i < n; ++i, j += SPLIT ? 2 : 1) {
      if (!mbar_wait_warp(bar.s_full(I), sc & 1, abort, p.flags, lim)) return;
      if (live) {
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
        const bool masked = L - j * BN < BN;
        if (masked) {
          if (!have_mask &&
              !mbar_wait_warp(bar.tree_full(b), (mc >> 1) & 1, abort, p.flags, lim))
            return;
          have_mask = true;
          int a = node;
#pragma unroll
          for (int c = 3; c >= 0; --c) {
            const uint32_t bits = seen_bits(trees[b], a, j * BN - L + 32 * c);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1u)) s[32 * c + e] = -INFINITY;
          }
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
        if (i > 0 && __any_sync(0xffffffffu, grow)) {
          // O_I already holds the chain's earlier tiles (S_I was issued after their products
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
        // (one copy of this code for all tiles, as the roles share one instruction cache: with one
        // for masked tiles beside it, 200 nodes take 234 us instead of 219)
        write_p<false>(s, sl2, ms, lane_base + C::p_col(I), sum);
        l += (sum[0].x + sum[1].x) + (sum[0].y + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
      }
      mbar_arrive(bar.p_full(I));
      ++sc;
    }
    bool bad = false;
    if (FIELD(x, tail)) {
      // (every warp meets every mask, so that none is a buffer ahead)
      if (!have_mask && !mbar_wait_warp(bar.tree_full(b), (mc >> 1) & 1, abort, p.flags, lim)) return;
      bad |= bad_trees[b] != 0;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar.tree_empty(b));
      ++mc;
    }

    // ---- results of the piece: O and LSE, or a partial output ----
    const int slot = FIELD(x, slot), pair_now = FIELD(x, pair), last = FIELD(x, last);
    const int head = place() >> 8, at = (2 * pair_now + (SPLIT ? 0 : I)) * w.tile_nodes + (place() & 255);
    const bool dead = node < 0;
    const bool exists = at < p.Tn && head < w.group && pair_now < w.pairs;
    // a row tile without nodes: zeros (or NaN), once
    const bool computed = SPLIT ? total > 0 : n > 0;
    const bool whole = computed ? slot < 0 : true;
    const bool write = exists && (computed || last);
    float f0 = 0.f, f1 = 0.f;         // factors of O_0 and O_1 (one of them without SPLIT)
    float M = m, sum = l;
    bool two = false;
    // the chain's last P V product
    if (n > 0 && !mbar_wait_warp(bar.s_free(I), (sc - 1) & 1, abort, p.flags, lim)) return;
    tc_fence_after();
    if (SPLIT && total > 0) {
      two = total > 1;  // (chain 1 has a tile)
      join[I * BM + tile_row] = make_float2(m, l);
      if (!meet(0)) return;
      const float2 a = join[tile_row], c = join[BM + tile_row];  // (-inf, 0 without a tile)
      M = fmaxf(a.x, c.x);
      const float Ms = M == -INFINITY ? 0.f : M;
      f0 = ex2((a.x - Ms) * sl2);
      f1 = ex2((c.x - Ms) * sl2);
      sum = f0 * a.y + f1 * c.y;
    } else {
      f0 = 1.f;
    }
    const bool none = sum == 0.f || dead || !computed;  // no key is seen (a NaN is a result)
    const bool nan = FIELD(x, bad) != 0 || (bad && !dead);
    const float inv = nan ? kNan : (none ? 0.f : 1.f / sum);
    const float lse = nan ? kNan : (none ? -INFINITY : M * p.scale + logf(sum));
    f0 *= inv;
    f1 *= inv;
    const size_t out_row =
        (static_cast<size_t>(FIELD(x, r)) * p.Hq + FIELD(x, kvh) * w.group + head) * p.Tn + at;
    const int unit_row = (SPLIT ? 0 : BM * I) + tile_row;
    const size_t part = static_cast<size_t>(max(slot, 0)) * w.unit_rows;
    // SPLIT: each warpgroup writes half of the channels
    constexpr int COLS = SPLIT ? D / 2 : D;
    const int c0 = SPLIT ? COLS * I : 0;
    const bool has_o = live && computed;
    if (__any_sync(0xffffffffu, write)) {
#pragma unroll 1
      for (int c = c0; c < c0 + COLS; c += 16) {
        uint32_t o[16], o1[16];
        if (has_o) {
          tmem_ld16(lane_base + C::o_col(SPLIT ? 0 : I) + c, o);
          if (SPLIT && two) tmem_ld16(lane_base + C::o_col(1) + c, o1);
          tmem_wait_ld();
          reg_fence16(o);
          if (SPLIT && two) reg_fence16(o1);
        }
        float f[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          f[e] = has_o && !none ? __uint_as_float(o[e]) * f0 : inv;  // (zero, or NaN)
          if (SPLIT && two && has_o && !none) f[e] = fmaf(__uint_as_float(o1[e]), f1, f[e]);
        }
        if (write && whole) {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + out_row * D + c);
#pragma unroll
          for (int v = 0; v < 2; ++v)
            dst[v] = make_uint4(pack_bf16x2(f[8 * v], f[8 * v + 1]), pack_bf16x2(f[8 * v + 2], f[8 * v + 3]),
                                pack_bf16x2(f[8 * v + 4], f[8 * v + 5]),
                                pack_bf16x2(f[8 * v + 6], f[8 * v + 7]));
        } else if (write) {
          float4* dst = reinterpret_cast<float4*>(w.part_o + part * D) + (c / 4) * w.unit_rows + unit_row;
#pragma unroll
          for (int v = 0; v < 4; ++v)
            dst[v * w.unit_rows] = make_float4(f[4 * v], f[4 * v + 1], f[4 * v + 2], f[4 * v + 3]);
        }
      }
    }
    if (write && (!SPLIT || I == 0)) {
      if (!whole)
        w.part_lse[part + unit_row] = lse;
      else if (p.lse != nullptr)
        p.lse[out_row] = lse;
    }
    // the next piece's products may overwrite what the other warpgroup reads here
    if (SPLIT && total > 0) {
      if (!meet(1)) return;
      ++jc;
    }
  }
}

// This CTA's range of the steps, found by all threads together (a request a thread).
__device__ void make_plan(const Work& w, Plan* plan, int* sums) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto block_sum = [&](int v) {  // over all threads, in every thread
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) sums[warp] = v;
    __syncthreads();
    int t = 0;
    for (int i = 0; i < kThreads / 32; ++i) t += sums[i];
    return t;
  };
  // of a KV head: rounds with nodes, the last of which may cost less, then those without
  auto line = [&](const Sizes& z) {
    int sum = 0;
    for (int i = 0; i < w.rounds; ++i) sum += kSegCost + steps_of(w, z, i) * step_cost(w, z, i);
    return sum;
  };
  auto line_at = [&](int r) { return r < w.p.S ? line(sizes_of(w.p, r)) * w.p.Hkv : 0; };
  const int first = line_at(threadIdx.x);  // (the only requests, usually)
  int mine = first;
  for (int r = threadIdx.x + kThreads; r < w.p.S; r += kThreads) mine += line_at(r);
  const int total = block_sum(mine);
  const int W = max(1, min(static_cast<int>(gridDim.x) / w.team, total / kMostCost));
  const int k = blockIdx.x / w.team;
  const int share = total / W, extra = total - share * W;  // the first `extra` take one more
  const int lo = k < W ? k * share + min(k, extra) : total;
  const int hi = k < W ? lo + share + (k < extra ? 1 : 0) : total;
  if (threadIdx.x == 0) *plan = Plan{lo, hi, hi, 0, 0, 0, share, extra};
  int before = 0;
  for (int r0 = 0; r0 < w.p.S && lo < hi; r0 += kThreads) {
    const int r = r0 + threadIdx.x;
    const int own = r0 == 0 ? first : line_at(r);
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += v;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    int all = 0;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) incl += sums[i];
      all += sums[i];
    }
    incl += before;
    if (own > 0 && incl - own <= lo && lo < incl) {
      // the first step at or behind lo
      Sizes z = sizes_of(w.p, r);
      const int head = own / w.p.Hkv, kvh = (lo - (incl - own)) / head;
      int pos = incl - own + kvh * head, round = 0;
      while (round + 1 < w.rounds) {
        const int len = kSegCost + steps_of(w, z, round) * step_cost(w, z, round);
        if (pos + len > lo) break;
        pos += len;
        ++round;
      }
      pos += kSegCost;
      const int steps = steps_of(w, z, round), cost = step_cost(w, z, round);
      int j = lo > pos ? (lo - pos + cost - 1) / cost : 0, rr = r, s = kvh * w.rounds + round;
      if (j < steps) {
        pos += j * cost;
      } else {  // behind the last one: the next segment's first
        pos += steps * cost + kSegCost;
        j = 0;
        if (++s == w.segs) {
          s = 0;
          ++rr;
        }
      }
      plan->pos = rr < w.p.S ? pos : hi;
      plan->r = rr;
      plan->s = s;
      plan->j = j;
    }
    before += all;
    if (before > lo) break;  // (the same in every thread)
  }
}

template <int D, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Work w) {
  using C = Cfg<D, SPLIT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const Bars<D, SPLIT> bar{sbase + C::OFF_BAR};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::OFF_MISC + 4);
  Plan* plan_at = reinterpret_cast<Plan*>(smem + C::OFF_PLAN);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the merge kernel (or what else follows as a programmatic dependent) waits for this
  // grid's results
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (sbase - raw > C::SLACK) {  // (the declaration asks for it)
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (threadIdx.x == 0) {
      raise_flag(w.p.flags, DEVFLAG_TIMEOUT);
      if (!w.direct) w.cut[blockIdx.x].pieces = 0;
    }
    return;
  }
  if (threadIdx.x == 0) {
    mbar_init(bar.q_full(), 1);
    mbar_init(bar.q_empty(), 1);
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(bar.slot_full(s), 1);
      mbar_init(bar.slot_empty(s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar.s_full(i), 1);
      mbar_init(bar.s_free(i), 1);
      mbar_init(bar.p_full(i), 128);
      mbar_init(bar.tree_full(i), 1);
      mbar_init(bar.tree_empty(i), 8);
      mbar_init(bar.joined(i), 256);
    }
    for (int i = 0; i < kPieces; ++i) {
      mbar_init(bar.piece_full(i), 1);
      mbar_init(bar.piece_empty(i), kRoles);
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
  // the preceding kernel's writes (an append's) are complete and visible past this point
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (!w.direct) make_plan(w, plan_at, reinterpret_cast<int*>(smem + C::OFF_SUMS));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < 4) {
    regs_decrease<regs_wg0(SPLIT)>();
    if (warp == 0) {
      producer_warp<D, SPLIT>(&tmQ, &tmK, &tmV, w, sbase, bar, abort);
    } else if (warp == 1) {
      MmaWarp<D, SPLIT> mma(w, bar, abort, sbase, tmem);
      mma.run();
      // Every product this warp issued has finished once the teardown barrier flips.
      mma_commit_warp(bar.teardown());
      if (lane == 0) mbar_wait_quiet(bar.teardown(), 0, 1000000000ull);
      __syncwarp();
    } else if (warp == 2) {
      tree_warp<D, SPLIT>(w, smem, bar, abort);
    } else if (lane == 0) {
      // (the plan is not set, nor read, if w.direct)
      planner_warp<D, SPLIT>(w, *plan_at, smem, bar, abort);
    }
  } else {
    regs_increase<regs_softmax(SPLIT)>();
    softmax_wg<D, SPLIT>(w, smem, tmem, bar, abort, warp < 8 ? 0 : 1);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// LSE = M + ln sum_j e^{LSE_j - M}, O = sum_j e^{LSE_j - LSE} O_j over the pieces of a cut
// segment: a thread 8 channels of a row, the lanes of a warp neighbouring rows, N pieces in
// flight.  Bound by latencies: 3 us on 64 requests x 8 nodes (15 MB of partial outputs), 10 on 8 x
// 200 nodes (39 MB).  A warp a row, its lanes side by side in the channels, with scattered stores
// of the partial outputs: 13 us on the latter; 16 channels a thread no faster.
constexpr int kMergeThreads = 128;
template <int D, int N>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ Work w) {
  constexpr int PARTS = D / 8;
  constexpr float kLog2e = 1.4426950408889634f;
  // launched as a programmatic dependent: the results are complete and visible past this
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int row_groups = (w.unit_rows + 31) / 32;
  const int unit = blockIdx.y * (kMergeThreads / 32) + (threadIdx.x >> 5);  // (row group, part)
  const int part = unit / row_groups, unit_row = (unit - part * row_groups) * 32 + (threadIdx.x & 31);
  const int tile = unit_row / BM, tile_row = unit_row - tile * BM;
  const int tile_node = (tile_row * w.per_group) >> 16, head = tile_row - tile_node * w.group;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = w.cut[blockIdx.x];
  const int node = (2 * cut.pair + tile) * w.tile_nodes + tile_node;
  // (a row tile without nodes has been written already)
  if (cut.pieces <= 0 || part >= PARTS || unit_row >= w.unit_rows || tile >= cut.tiles ||
      tile_node >= w.tile_nodes || node >= w.p.Tn)
    return;
  float m = -INFINITY, sum = 0.f, o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  for (int j = 0; j < cut.pieces; j += N) {
    float lse[N];
    float4 v[N][2];
#pragma unroll
    for (int s = 0; s < N; ++s) {
      lse[s] = -INFINITY;
      v[s][0] = v[s][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (j + s < cut.pieces) {
        const int slot = j + s == 0 ? cut.slot : 2 * (static_cast<int>(blockIdx.x) + (j + s) * w.team);
        const size_t at = static_cast<size_t>(slot) * w.unit_rows;
        lse[s] = w.part_lse[at + unit_row];
        const float4* src = reinterpret_cast<const float4*>(w.part_o + at * D) + unit_row;
        v[s][0] = src[2 * part * w.unit_rows];
        v[s][1] = src[(2 * part + 1) * w.unit_rows];
      }
    }
    float mn = m;
#pragma unroll
    for (int s = 0; s < N; ++s) mn = fmaxf(mn, lse[s]);
    const float ms = mn == -INFINITY ? 0.f : mn;
    const float al = ex2((m - ms) * kLog2e);
    m = mn;
    sum *= al;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= al;
#pragma unroll
    for (int s = 0; s < N; ++s) {
      const float f = ex2((lse[s] - ms) * kLog2e);
      sum += f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        o[4 * h] = fmaf(f, v[s][h].x, o[4 * h]);
        o[4 * h + 1] = fmaf(f, v[s][h].y, o[4 * h + 1]);
        o[4 * h + 2] = fmaf(f, v[s][h].z, o[4 * h + 2]);
        o[4 * h + 3] = fmaf(f, v[s][h].w, o[4 * h + 3]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;  // (no key is seen)
  const size_t out =
      (static_cast<size_t>(cut.r) * w.p.Hq + cut.kvh * w.group + head) * w.p.Tn + node;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(w.p.o) + out * D + 8 * part) =
      make_uint4(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv),
                 pack_bf16x2(o[4] * inv, o[5] * inv), pack_bf16x2(o[6] * inv, o[7] * inv));
  if (w.p.lse != nullptr && part == 0) w.p.lse[out] = sum == 0.f ? -INFINITY : m + logf(sum);
}

struct Shape {
  int group, tile_nodes, row_tiles, pairs, team, rounds, segs, unit_rows;
  long long units, steps;  // segments of the batch, and their steps at most
  bool small;   // for tree_short.cu
  bool direct;  // CTAs take whole segments
};

Shape shape_of(int S, int Tn, int Hq, int Hkv, int max_seq_len) {
  Shape s;
  s.group = Hq / Hkv;
  s.tile_nodes = tree_tile_nodes(s.group, Tn);
  s.row_tiles = (Tn + s.tile_nodes - 1) / s.tile_nodes;
  s.pairs = (s.row_tiles + 1) / 2;
  s.rounds = tree_rounds(s.group, Tn);
  s.team = (s.pairs + s.rounds - 1) / s.rounds;
  s.segs = Hkv * s.rounds;
  s.unit_rows = s.row_tiles == 1 ? s.tile_nodes * s.group : 2 * BM;
  const long long per_seg = std::max<long long>(1, (max_seq_len + (BN - 1ll)) / BN);
  s.units = static_cast<long long>(S) * s.segs;
  s.steps = per_seg * s.units;
  // Which kernel, by the bound on the keys.  Device time in us, tree_short.cu / whole segments / cut
  // segments (batches: lengths from half the bound to it; one request: as long as the bound; D 128
  // but for *):
  //   requests x heads   rows  100               250               500               800               1200              1800
  //   1 x 8/2 *            20  4.4 / 6.9 / 13    6.0 / 7.5 / 9.9   9.1 / 9.6 / 11    13 / 12 / 11      18 / 16 / 11      26 / 20 / 12
  //   1 x 32/8             16  5.6 / 8.2 / 14    7.8 / 8.9 / 14    12 / 12 / 12      17 / 16 / 14      23 / 20 / 14      33 / 28 / 14
  //   1 x 32/8             32  7.1 / 8.2 / 14    9.4 / 8.9 / 14    14 / 12 / 12      20 / 16 / 14      27 / 20 / 14      39 / 28 / 15
  //   1 x 12/2             48  6.6 / 8.0 / 14    10 / 8.7 / 11     17 / 12 / 12      26 / 16 / 13      36 / 20 / 13      54 / 28 / 13
  //   5 x 12/2             48  7.8 / 8.2 / 14    10 / 8.9 / 14     18 / 12 / 14      26 / 16 / 14      36 / 20 / 14      53 / 26 / 15
  //   20 x 32/8            32  9.5 / 12 / 15     13 / 14 / 18      18 / 18 / 21      24 / 24 / 25      30 / 25 / 27      44 / 41 / 33
  //   64 x 12/2            48  9.4 / 9.1 / 15    14 / 11 / 17      21 / 13 / 19      31 / 18 / 23      42 / 22 / 25      60 / 28 / 29
  //   100 x 16/8           64  27 / 32 / 38      38 / 42 / 53      55 / 54 / 71      75 / 70 / 85      103 / 89 / 97     142 / 124 / 115
  //   100 x 16/8 *          8  9 / 28 / 32       14 / 32 / 38      21 / 43 / 59      29 / 52 / 74      39 / 65 / 84      54 / 88 / 96
  //   200 x 8/2            16  9 / 17 / 20       14 / 21 / 26      20 / 31 / 37      27 / 39 / 45      37 / 52 / 51      52 / 71 / 62
  // The rule takes the better one but for one request of 32 rows (250 keys: 9.4 where whole segments
  // take 8.9, 500: 14 and 12) and 64 requests of 48 (100 keys: 9.4 and 9.1; 1800: 29 and 28).  At its
  // own edge, one request of 16 rows and 768 keys takes 16 where cut segments take 14.
  const int rows = s.group * Tn;
  const long long heads = static_cast<long long>(S) * Hkv;
  const bool many = heads >= 304;  // two a SM
  if (rows <= 16)
    s.small = per_seg <= 6 || (many && per_seg <= 20);
  else if (rows <= 32)
    s.small = per_seg <= 4;
  else
    s.small = rows <= kTreeShortRows && (per_seg <= 1 || (many && per_seg <= 4));
  s.direct = s.small || per_seg <= 6 || (s.units >= 100 && per_seg <= 10);
  return s;
}

// CTAs of a launch: the workspace is laid out for as many on every device, so that it depends on
// the sizes alone.
constexpr int kMaxGrid = 160;
int grid_of(const Shape& s, int num_sms) {
  const int teams = std::max(1, std::min(num_sms, kMaxGrid) / s.team);
  return s.team * static_cast<int>(std::min<long long>(teams, s.direct ? s.units : s.steps));
}

struct Layout {
  size_t off_lse, off_cut, bytes;  // part_o at 0
};
Layout layout_of(const Shape& s, int D) {
  Layout l{};
  if (s.direct) return l;
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t grid = static_cast<size_t>(grid_of(s, kMaxGrid));
  const size_t rows = 2 * grid * s.unit_rows;
  l.off_lse = up(rows * D * sizeof(float));
  l.off_cut = l.off_lse + up(rows * sizeof(float));
  l.bytes = l.off_cut + up(grid * sizeof(Cut));
  return l;
}

template <int D, bool SPLIT>
cudaError_t launch(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                   const Work& w, int grid, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Cfg<D, SPLIT>::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, tree_attn_kernel<D, SPLIT>, tmQ, tmK, tmV, w);
  if (e != cudaSuccess || w.direct) return e;
  cfg.gridDim = dim3(grid, ((w.unit_rows + 31) / 32 * (D / 8) + kMergeThreads / 32 - 1) / (kMergeThreads / 32));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  // (few segments are cut into many pieces each)
  const long long units = static_cast<long long>(w.p.S) * w.segs * w.team;
  return grid > 4 * units ? cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 8>, w)
                          : cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, 2>, w);
}

template <int D, bool SPLIT>
cudaError_t set_smem() {
  return cudaFuncSetAttribute(tree_attn_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (Cfg<D, SPLIT>::SMEM_BYTES));
}

}  // namespace

int tree_tile_nodes(int group, int Tn) { return std::min(BM / group, Tn); }
int tree_rounds(int group, int Tn) {
  if (Tn <= 0) return 0;
  const int nodes = tree_tile_nodes(group, Tn), pairs = ((Tn + nodes - 1) / nodes + 1) / 2;
  return (pairs + kMaxTeam - 1) / kMaxTeam;
}

size_t tree_attn_workspace_bytes(int S, int Tn, int Hq, int Hkv, int D, int max_seq_len) {
  return layout_of(shape_of(S, Tn, Hq, Hkv, max_seq_len), D).bytes;
}

cudaError_t prepare_tree_attn() {
  cudaError_t e;
  if ((e = prepare_tree_short()) != cudaSuccess) return e;
  if ((e = set_smem<64, true>()) != cudaSuccess) return e;
  if ((e = set_smem<64, false>()) != cudaSuccess) return e;
  if ((e = set_smem<128, true>()) != cudaSuccess) return e;
  return set_smem<128, false>();
}

cudaError_t launch_tree_attn(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                             const TreeParams& p, void* workspace, int num_sms,
                             cudaStream_t stream) {
  const Shape s = shape_of(p.S, p.Tn, p.Hq, p.Hkv, p.max_seq_len);
  if (s.small) return launch_tree_short(tmK, tmV, p, stream);
  const Layout l = layout_of(s, p.D);
  char* ws = static_cast<char*>(workspace);
  Work w{};
  w.p = p;
  w.part_o = reinterpret_cast<float*>(ws);
  w.part_lse = reinterpret_cast<float*>(ws + l.off_lse);
  w.cut = reinterpret_cast<Cut*>(ws + l.off_cut);
  w.group = s.group;
  w.per_group = (65536 + s.group - 1) / s.group;
  w.tile_nodes = s.tile_nodes;
  w.pairs = s.pairs;
  w.team = s.team;
  w.rounds = s.rounds;
  w.segs = s.segs;
  w.unit_rows = s.unit_rows;
  w.direct = s.direct;
  const int grid = grid_of(s, num_sms);
  const bool split = s.row_tiles == 1;
  if (p.D == 64)
    return split ? launch<64, true>(tmQ, tmK, tmV, w, grid, stream)
                 : launch<64, false>(tmQ, tmK, tmV, w, grid, stream);
  return split ? launch<128, true>(tmQ, tmK, tmV, w, grid, stream)
               : launch<128, false>(tmQ, tmK, tmV, w, grid, stream);
}

}  // namespace gbattn
