// draft_verify.cu -- which drafted tokens the target model accepts, from given random
// numbers, and the token after them.
//
// At a node with the target's row p and the draft's row q (from which its children were
// drawn independently), with w = p, W = 1: child x stands if u q(x) W < w(x), i.e. with
// probability min(1, (w(x) / W) / q(x)).  When it falls, w becomes max(w - W q, 0) and W
// its sum: w / W is the distribution that what is still to be drawn has to follow (the
// residual), kept without divisions.  The last token is drawn from w by where u times its
// sum falls in the running sum.
//
// A token hangs on which side of a border a random number lies, so sums must not depend on
// an order and must be finer than fp32: they are sums of integers, which are exact in any
// order.  A test of a token takes probabilities as multiples of 2^-62 (an fp32 from 2^-38 up
// exactly) and products in 128 bits.  Sums over a row take the exact p, or max(p - q, 0), rounded
// to a multiple of 2^-44 (5e-9 of a distribution over 2^17 tokens at the very most, 1e-11 as
// roundings go): adding 2 to an fp32 below 1 and taking it off again rounds it to 2^-22,
// what is left over goes the same way to 2^-44, and the bits of the two sums are the integers
// to be added up.  That is 13 instructions a token, half of them on pairs; integers made by shifts take 45 (64
// requests x 8 drafts, 131072 tokens: 104 us), the compiler's conversions to 64 bits, which run at the
// rate of 64-bit floating point, more yet (159).
//
// A cluster of CTAs takes a request.  CTA 0 leads: it reads the tree and, for all nodes at
// once, the two probabilities that a test of the node would need, and walks down the tree
// in registers and shared memory.  Only where a child falls, or at the end, all V values of
// a row (or two) are needed: CTA c then sums tokens [c chunk, (c + 1) chunk), a warp a tile
// of them at a time, keeps the tiles' sums, and puts its sum into every CTA's shared memory.
// The leader tells the others what to do next, so the control flow, and with it the number
// of cluster barriers that each CTA meets, is decided in one place.  The last token's CTA is found from the CTAs' sums,
// its tile from the tiles' sums, and only that tile is read again.
#include <cuda_runtime.h>

#include <cstring>

#include "gbattn.h"
#include "ptx.cuh"
#include "tree.h"

namespace gbattn {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxNodes = GBATTN_TREE_MAX_NODES;
static_assert(kThreads == kMaxNodes, "a thread a node");
constexpr int kMaxCtas = 16;   // of a cluster
constexpr int kPerLane = 16;   // values of a row that a lane reads at once
constexpr int kSpan = 32 * kPerLane;
constexpr int kMaxTiles = 256;
constexpr int kMaxKept = 16384;  // tokens of a CTA whose w is kept from fall to fall (128 KB)
static_assert(kMaxKept % kSpan == 0, "whole spans");

using u64 = unsigned long long;
constexpr u64 kOne = 1ull << 62;

// A probability (or random number) as a multiple of 2^-62; NaN and negative values are 0.
// The significand goes to the top of 64 bits and down by the exponent (PTX shifts by 32 and
// more give 0; the compiler's conversion to 64 bits runs at the rate of 64-bit floating point).
__device__ __forceinline__ u64 fixed(float v) {
  const uint32_t bits = __float_as_uint(__saturatef(v));
  const uint32_t m = (bits << 8) | 0x80000000u, e = bits >> 23;  // v = m 2^(e - 158)
  uint32_t hi, up, down;
  asm("shr.u32 %0, %1, %2;" : "=r"(hi) : "r"(m), "r"(128u - e));
  asm("shl.b32 %0, %1, %2;" : "=r"(up) : "r"(m), "r"(e - 96u));
  asm("shr.u32 %0, %1, %2;" : "=r"(down) : "r"(m), "r"(96u - e));
  return static_cast<u64>(hi) << 32 | (up | down);
}
__device__ __forceinline__ float value(float v) { return v; }
__device__ __forceinline__ float value(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// q W for a probability q, rounded down: the 32-bit significand times W, down by the exponent.
__device__ __forceinline__ u64 product(float q, u64 W) {
  const uint32_t bits = __float_as_uint(__saturatef(q));
  const uint32_t m = (bits << 8) | 0x80000000u, e = bits >> 23;
  const u64 low = static_cast<u64>(m) * static_cast<uint32_t>(W);
  const u64 high = static_cast<u64>(m) * static_cast<uint32_t>(W >> 32) + (low >> 32);
  u64 r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(high), "r"(126u - e));  // (by 64 and more: 0)
  return e == 127u ? W : r;
}
__device__ __forceinline__ u64 minus(u64 a, u64 b) { return a > b ? a - b : 0; }
// a b 2^-62, rounded down.
__device__ __forceinline__ u64 share_of(u64 a, u64 b) { return (__umul64hi(a, b) << 2) | ((a * b) >> 62); }
// Whether a b 2^-62 < c, exactly.
__device__ __forceinline__ bool product_below(u64 a, u64 b, u64 c) {
  const u64 hi = __umul64hi(a, b), lo = a * b;
  return hi < c >> 2 || (hi == c >> 2 && lo < c << 62);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_prefix(u64 v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Address of this CTA's shared variable in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t remote(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void store_remote(uint32_t a, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(v) : "memory");
}

// What the leader has the cluster do.  kRest: sum of what is left once W q is taken off, and
// kept as there is another child to try; kRestLast: there is none.
enum : int { kDone, kScan, kRest, kRestLast, kDraw };
struct Command {
  int op, node, level, count;
  u64 total;  // kRest: W; kDraw: where the random number falls in the running sum
};
static_assert(sizeof(Command) == 24, "three words");

// w of one token after `level` falls, and less W q if `rest`.
__device__ __forceinline__ u64 left(float p, float q, const u64* W, int level, bool rest) {
  u64 w = fixed(p);
  const int n = level + (rest ? 1 : 0);
  for (int i = 0; i < n; ++i) w = minus(w, i == 0 ? fixed(q) : product(q, W[i]));  // W[0] = 1
  return w;
}

// The sums' form of values in [0, 1]: hi 2^-22 + lo 2^-44 (added up modulo 2^32, with an offset
// for each value).
struct Halves {
  uint32_t hi, lo;
};
constexpr uint32_t kHiOffset = 0x40000000u, kLoOffset = 0x35400000u;  // 2, 1.5 x 2^-21
__device__ __forceinline__ u64 whole(Halves h, uint32_t n) {  // of n values, as a multiple of 2^-62
  const long long hi = h.hi - n * kHiOffset;                  // (below 2^31: n <= 256)
  const int lo = static_cast<int>(h.lo - n * kLoOffset);
  return static_cast<u64>((hi << 22) + lo) << 18;
}
// Of d + e for a pair of values, |e| half a unit of d's last place at most.
__device__ __forceinline__ void halves(float2 d, float2 e, Halves& x, Halves& y) {
  const float2 t = __fadd2_rn(d, make_float2(2.f, 2.f));
  const float2 back = __fadd2_rn(t, make_float2(-2.f, -2.f));
  const float2 r = __fadd2_rn(d, make_float2(-back.x, -back.y));  // exact
  const float2 u = __fadd2_rn(__fadd2_rn(r, e), make_float2(0x1.8p-21f, 0x1.8p-21f));
  x = Halves{__float_as_uint(t.x), __float_as_uint(u.x)};
  y = Halves{__float_as_uint(t.y), __float_as_uint(u.y)};
}
// Of max(p - q, 0): where p > q, p - q is d + e exactly.
__device__ __forceinline__ void rest_halves(float2 p, float2 q, Halves& x, Halves& y) {
  p = make_float2(__saturatef(p.x), __saturatef(p.y));
  q = make_float2(-__saturatef(q.x), -__saturatef(q.y));
  float2 d = __fadd2_rn(p, q);
  float2 e = __fadd2_rn(__fadd2_rn(p, make_float2(-d.x, -d.y)), q);
  e = make_float2(d.x > 0.f ? e.x : 0.f, d.y > 0.f ? e.y : 0.f);
  halves(make_float2(fmaxf(d.x, 0.f), fmaxf(d.y, 0.f)), e, x, y);
}
__device__ __forceinline__ void prob_halves(float2 p, Halves& x, Halves& y) {
  halves(make_float2(__saturatef(p.x), __saturatef(p.y)), make_float2(0.f, 0.f), x, y);
}
// w of one token in that form, after `level` falls and less W q if `rest`.
__device__ __forceinline__ u64 left_rounded(float p, float q, const u64* W, int level, bool rest) {
  const int n = level + (rest ? 1 : 0);
  Halves x, y;
  if (n == 0)
    prob_halves(make_float2(p, 0.f), x, y);
  else
    rest_halves(make_float2(p, 0.f), make_float2(q, 0.f), x, y);
  u64 w = whole(x, 1);
  for (int i = 1; i < n; ++i) w = minus(w, product(q, W[i]));
  return w;
}

// kPerLane values of a row from `i` on, 32 apart; those from `end` on are 0.
template <typename T>
__device__ __forceinline__ void read_span(const T* row, int i, int end, bool all, float (&v)[kPerLane]) {
  if (all) {
    T x[kPerLane];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) x[k] = row[i + 32 * k];
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) v[k] = value(x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) v[k] = i + 32 * k < end ? value(row[i + 32 * k]) : 0.f;
  }
}

template <typename T, bool DRAWN>
__global__ void __launch_bounds__(kThreads) draft_verify_kernel(const VerifyParams p) {
  __shared__ int parent[kMaxNodes], token[kMaxNodes], path[kMaxNodes];
  __shared__ u64 chance[kMaxNodes];                    // u, p and q of every node
  __shared__ float pv[kMaxNodes], qv[kMaxNodes];
  __shared__ u64 W[kMaxNodes];           // sums of w by level
  __shared__ u64 sums[kMaxTiles];        // of this CTA's tiles
  __shared__ u64 totals[kMaxCtas];       // of all CTAs
  __shared__ u64 part[kWarps];
  __shared__ Command cmd;
  __shared__ u64 gone[DRAWN ? 1 : kMaxNodes], gone_w[DRAWN ? 1 : kMaxNodes];  // fallen tokens
  extern __shared__ u64 kept[];          // w of the CTA's first p.kept tokens, as of `held` falls
  const uint32_t ctas = cluster_size(), rank = cluster_rank();
  const int r = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  cluster_arrive();  // every CTA's shared memory may be written once all are past the wait
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const T* p_rows = static_cast<const T*>(p.p) + r * p.p_stride[0];
  const T* q_rows = DRAWN ? static_cast<const T*>(p.q) + r * p.q_stride[0] : nullptr;
  int n = 0;
  if (rank == 0) {
    n = p.tree_lens ? p.tree_lens[r] : p.Tn;
    const bool bad_n = n < 0 || n > p.Tn;
    if (bad_n) n = 0;
    const size_t row = static_cast<size_t>(r) * p.Tn;
    bool bad = false;
    if (tid < n) {
      const int up = p.parents[row + tid], x = p.tokens[row + tid];
      parent[tid] = up;
      token[tid] = x;
      chance[tid] = fixed(p.uniforms[row + tid]);
      bad = up < -1 || up >= tid;
      float a = 0.f, b = 0.f;
      if (!bad && up >= 0 && x >= 0 && x < p.V) {
        a = value(p_rows[up * p.p_stride[1] + x]);
        if (DRAWN) b = value(q_rows[up * p.q_stride[1] + x]);
      }
      pv[tid] = a;
      qv[tid] = DRAWN ? b : 1.f;
    }
    const bool bad_tree = __syncthreads_or(bad);
    if ((bad_n || bad_tree) && tid == 0) raise_flag(p.flags, bad_n ? DEVFLAG_BAD_SEQLEN : DEVFLAG_BAD_TREE);
    if (bad_tree) n = 0;
    if (tid == 0) path[0] = 0;
  }
  cluster_wait();

  // the leader's walk (warp 0 of CTA 0)
  int cur = 0, at = 0, level = 0, fallen = 0, count = n > 0 ? 1 : 0;
  u64 total = kOne;
  enum { kNothing, kRested, kSummed, kLast } waiting = kNothing;
  bool summed = false;  // the last sums are those of the present w
  int op = kDone, s_level = 0, s_node = 0;
  bool s_rest = false;
  int held = 0, held_node = -1;
  const int c0 = rank * p.chunk, c1 = min(p.V, c0 + p.chunk);  // (chunk * ctas < 2^31)

  for (;;) {
    if (rank == 0 && warp == 0) {
      Command next{kDone, cur, 0, count, 0};
      u64 all = 0;
      if (waiting != kNothing) {
        all = warp_sum(lane < static_cast<int>(ctas) ? totals[lane] : 0);
        summed = true;
        if (waiting == kRested) {
          if (all > 0) {
            total = all;
            ++level;
          } else {
            summed = false;
          }
        }
      }
      bool again = waiting == kSummed;  // child `at` has been found to fall already
      waiting = kNothing;
      if (n > 0) {
        for (;;) {
          if (!again) {
            // the next child of the node reached
            int found = -1;
            for (int b = (at + 1) & ~31; b < n && found < 0; b += 32) {
              const int i = b + lane;
              const unsigned hit = __ballot_sync(0xffffffffu, i > at && i < n && parent[i] == cur);
              if (hit) found = b + __ffs(hit) - 1;
            }
            if (found < 0) {
              next.op = summed ? kDraw : kScan;
              waiting = kLast;
              break;
            }
            at = found;
          }
          const float q = qv[at];
          u64 w = left(pv[at], q, W, DRAWN ? level : 0, false);
          if (!DRAWN) {
            const u64 x = static_cast<u64>(token[at]);
            bool hit = false;
            for (int i = lane; i < fallen; i += 32) hit |= gone[i] == x;
            if (__any_sync(0xffffffffu, hit)) w = 0;
          }
          if (!again && product_below(chance[at], product(q, total), w)) {
            if (lane == 0) path[count] = at;
            ++count;
            cur = at;
            level = fallen = 0;
            total = kOne;
            summed = false;
            continue;
          }
          if (DRAWN) {
            bool more = false;
            for (int b = at & ~31; b < n; b += 32)
              more |= b + lane > at && b + lane < n && parent[b + lane] == cur;
            next.op = __any_sync(0xffffffffu, more) ? kRest : kRestLast;
            waiting = kRested;
            break;
          }
          if (!summed) {
            next.op = kScan;
            waiting = kSummed;
            break;
          }
          // without a draft the token itself is what falls, in the sums' form
          again = false;
          if (w > 0) w = left_rounded(pv[at], 0.f, W, 0, false);
          u64 out = 0;
          for (int i = lane; i < fallen; i += 32) out += gone_w[i];
          all = warp_sum(lane < static_cast<int>(ctas) ? totals[lane] : 0) - warp_sum(out);
          if (all > w) {
            total = all - w;
            if (w > 0) {
              if (lane < static_cast<int>(ctas)) {
                store_remote(remote(&gone[fallen], lane), static_cast<u64>(token[at]));
                store_remote(remote(&gone_w[fallen], lane), w);
              }
              __syncwarp();
              ++fallen;
            }
          }
        }
      }
      next.node = cur;
      next.count = count;
      next.level = DRAWN ? level : fallen;
      next.total = total;
      if (next.op == kDraw) {
        all = warp_sum(lane < static_cast<int>(ctas) ? totals[lane] : 0);
        if (!DRAWN) {
          u64 out = 0;
          for (int i = lane; i < fallen; i += 32) out += gone_w[i];
          all -= warp_sum(out);
        }
        next.total = share_of(chance[0], all);
        if (all == 0) next.op = kDone;
        if (lane == 0 && all == 0) raise_flag(p.flags, DEVFLAG_NO_MASS);
      }
      if (lane < static_cast<int>(ctas)) {
        u64 words[3];
        memcpy(words, &next, sizeof words);
        const uint32_t to = remote(&cmd, lane);
#pragma unroll
        for (int i = 0; i < 3; ++i) store_remote(to + 8 * i, words[i]);
      }
    }
    cluster_arrive();
    cluster_wait();
    const Command c = cmd;
    op = c.op;
    if (op == kDone || op == kDraw) break;

    // ---- sums of this CTA's tokens ----
    s_level = DRAWN ? c.level : 0;
    s_node = c.node;
    s_rest = op == kRest || op == kRestLast;
    if (s_rest) {
      if (tid == 0) W[c.level] = c.total;
      __syncthreads();
    }
    const T* pr = p_rows + s_node * p.p_stride[1];
    const T* qr = DRAWN ? q_rows + s_node * p.q_stride[1] : nullptr;
    const int falls = DRAWN ? s_level + (s_rest ? 1 : 0) : 0;
    const bool go_on = DRAWN && s_level > 0 && held == s_level && held_node == s_node;
    const u64 total_w = c.total;
    u64 mine = 0;
    for (int t = warp; c0 + t * p.tile < c1; t += kWarps) {
      u64 sum = 0;
      const int end = min(c1, c0 + (t + 1) * p.tile);
      for (int b = c0 + t * p.tile; b < end; b += kSpan) {
        float a[kPerLane], d[kPerLane];
        const bool all = b + kSpan <= end, fits = DRAWN && b - c0 + kSpan <= p.kept;
        u64* row_kept = kept + (b - c0 + lane);
        if (falls == 0) {
          read_span(pr, b + lane, end, all, a);
          Halves s{0, 0};
#pragma unroll
          for (int k = 0; k < kPerLane; k += 2) {
            Halves x, y;
            prob_halves(make_float2(a[k], a[k + 1]), x, y);
            s.hi += x.hi + y.hi;
            s.lo += x.lo + y.lo;
          }
          sum += whole(s, kPerLane);
        } else if (falls == 1) {
          read_span(pr, b + lane, end, all, a);
          read_span(qr, b + lane, end, all, d);
          Halves s{0, 0};
          const bool keep = fits && op == kRest;
#pragma unroll
          for (int k = 0; k < kPerLane; k += 2) {
            Halves x, y;
            rest_halves(make_float2(a[k], a[k + 1]), make_float2(d[k], d[k + 1]), x, y);
            s.hi += x.hi + y.hi;
            s.lo += x.lo + y.lo;
            if (keep) {
              row_kept[32 * k] = whole(x, 1);
              row_kept[32 * k + 32] = whole(y, 1);
            }
          }
          sum += whole(s, kPerLane);
        } else if (go_on && fits) {
          read_span(qr, b + lane, end, all, d);
#pragma unroll
          for (int k = 0; k < kPerLane; ++k) {
            u64 w = row_kept[32 * k];
            if (s_rest) {
              w = minus(w, product(d[k], total_w));
              row_kept[32 * k] = w;
            }
            sum += w;
          }
        } else {
          read_span(pr, b + lane, end, all, a);
          read_span(qr, b + lane, end, all, d);
#pragma unroll
          for (int k = 0; k < kPerLane; ++k) {
            const u64 w = left_rounded(a[k], d[k], W, s_level, s_rest);
            if (fits) row_kept[32 * k] = w;
            sum += w;
          }
        }
      }
      sum = warp_sum(sum);
      if (lane == 0) sums[t] = sum;
      mine += sum;
    }
    if (falls > 1 || op == kRest) {
      held = falls;
      held_node = s_node;
    }
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      mine = warp_sum(lane < kWarps ? part[lane] : 0);
      if (lane < static_cast<int>(ctas)) store_remote(remote(&totals[rank], lane), mine);
    }
    cluster_arrive();
    cluster_wait();
  }

  // ---- results ----
  const Command c = cmd;
  const size_t row = static_cast<size_t>(r) * p.Tn;
  if (rank == 0) {
    for (int j = tid; j < p.Tn; j += kThreads) {
      p.path[row + j] = j < c.count ? path[j] : -1;
      if (op == kDone || j != c.count - 1)  // (the last token is written by its CTA)
        p.tokens_out[row + j] = j < c.count - 1 ? token[path[j + 1]] : -1;
    }
    if (tid == 0) p.counts[r] = c.count;
  }
  if (op != kDraw || warp != 0) return;
  // the CTA whose tokens the running sum passes c.total in
  const int n_gone = DRAWN ? 0 : c.level;
  u64 own = lane < static_cast<int>(ctas) ? totals[lane] : 0;
  for (int i = 0; i < n_gone; ++i)
    if (static_cast<int>(gone[i]) / p.chunk == lane) own -= gone_w[i];
  u64 upto = warp_prefix(own);
  const u64 begin = __shfl_sync(0xffffffffu, upto - own, rank);
  const u64 stop = __shfl_sync(0xffffffffu, upto, rank);
  if (c.total < begin || c.total >= stop) return;
  u64 rest = c.total - begin;
  // its tile
  const int tiles = (c1 - c0 + p.tile - 1) / p.tile;
  int t = -1;
  for (int b = 0; b < tiles && t < 0; b += 32) {
    u64 s = b + lane < tiles ? sums[b + lane] : 0;
    for (int i = 0; i < n_gone; ++i) {
      const int x = static_cast<int>(gone[i]) - c0;
      if (x >= 0 && x < p.chunk && x / p.tile == b + lane) s -= gone_w[i];
    }
    const u64 incl = warp_prefix(s);
    const unsigned hit = __ballot_sync(0xffffffffu, rest < incl);
    if (hit) {
      t = b + __ffs(hit) - 1;
      rest -= __shfl_sync(0xffffffffu, incl - s, __ffs(hit) - 1);
    } else {
      rest -= __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  // its token: a lane's values are neighbours
  const T* pr = p_rows + s_node * p.p_stride[1];
  const T* qr = DRAWN ? q_rows + s_node * p.q_stride[1] : nullptr;
  const bool both = DRAWN && (s_rest || s_level > 0);
  const int end = min(c1, c0 + (t + 1) * p.tile);
  for (int b = c0 + t * p.tile; t >= 0 && b < end; b += kSpan) {
    u64 w[kPerLane], sum = 0;
    const int i0 = b + kPerLane * lane;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      w[k] = 0;
      if (i0 + k < end) {
        w[k] = left_rounded(value(pr[i0 + k]), both ? value(qr[i0 + k]) : 0.f, W, DRAWN ? s_level : 0,
                            DRAWN && s_rest);
        for (int i = 0; i < n_gone; ++i)
          if (gone[i] == static_cast<u64>(i0 + k)) w[k] = 0;
      }
      sum += w[k];
    }
    const u64 incl = warp_prefix(sum);
    const unsigned hit = __ballot_sync(0xffffffffu, rest < incl);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        u64 s = incl - sum;
        int x = i0 + kPerLane - 1;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {
          const bool before = s <= rest;
          s += w[k];
          if (before && s > rest) x = i0 + k;
        }
        p.tokens_out[row + c.count - 1] = x;
      }
      return;
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <typename T, bool DRAWN>
cudaError_t launch(const VerifyParams& p, int ctas, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.S) * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.kept * sizeof(u64);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, draft_verify_kernel<T, DRAWN>, p);
}

}  // namespace

cudaError_t prepare_draft_verify() {
  cudaError_t e = cudaSuccess;
  auto set = [&](const void* fn) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKept * sizeof(u64));
  };
  set(reinterpret_cast<const void*>(draft_verify_kernel<float, false>));
  set(reinterpret_cast<const void*>(draft_verify_kernel<float, true>));
  set(reinterpret_cast<const void*>(draft_verify_kernel<uint16_t, false>));
  set(reinterpret_cast<const void*>(draft_verify_kernel<uint16_t, true>));
  return e;
}

cudaError_t launch_draft_verify(VerifyParams p, bool bf16, int num_sms, cudaStream_t stream) {
  if (p.S <= 0) return cudaSuccess;
  int ctas = kMaxCtas;
  while (ctas > 1 && p.V <= ctas / 2 * kSpan * kWarps) ctas /= 2;
  auto up = [](long long x, long long m) { return (x + m - 1) / m * m; };
  const long long share = (static_cast<long long>(p.V) + ctas - 1) / ctas;
  p.tile = static_cast<int>(up((share + kMaxTiles - 1) / kMaxTiles, kSpan));
  p.chunk = static_cast<int>(up(share, p.tile));
  p.kept = p.q ? (p.chunk < kMaxKept ? p.chunk : kMaxKept) : 0;
  if (bf16)
    return p.q ? launch<uint16_t, true>(p, ctas, stream) : launch<uint16_t, false>(p, ctas, stream);
  return p.q ? launch<float, true>(p, ctas, stream) : launch<float, false>(p, ctas, stream);
}

}  // namespace gbattn
