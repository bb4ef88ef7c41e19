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
// After several falls w is still one subtraction from p,
//   w = max(p - A q, 0),  A = 1 + W_1 + W_2 + ..   (the W of the falls before),
// as a value that has become 0 stays 0 and the others have only been subtracted from.  So a
// sum over a row reads p and q and nothing else, whatever came before.
//
// A token hangs on which side of a border a random number lies, so sums must not depend on
// an order and must be finer than fp32: they are sums of integers, which are exact in any
// order.  A test of a token takes probabilities as multiples of 2^-62 (an fp32 from 2^-38 up
// exactly) and products in 128 bits.  Sums over a row take max(p - A q, 0), computed as the sum
// of two fp32, rounded to a multiple of 2^-44 (off by 0.5 of that for A = 0 and else by less than
// 0.88, see left_halves; 8e7 random tokens came to 0.67.  Roundings of 2^17 tokens add up to 1e-11
// as they go, 7e-9 at the very most): adding 2 to an fp32 below 1 and taking it off again rounds it to
// 2^-22, what is left over goes the same way to 2^-44, and the bits of the two sums are the
// integers to be added up.  That is some 16 instructions a token, most of them on pairs.  (Integers
// made by shifts take three times as many, and the first kernel, with the compiler's conversions
// to 64 bits and falls applied one after another, 159 us where this one takes 41.)
//
// A cluster of CTAs takes a request.  CTA 0 reads the tree and, for all nodes at once, the two
// probabilities that a test of the node would need, and writes them into the others' shared
// memory; every CTA then walks down the tree for itself, from the same data to the same
// decisions.  Only where a child falls, or at the end, all V values of a row (or two) are
// needed: CTA c then sums tokens [c chunk, (c + 1) chunk), a warp a tile of them at a time, keeps
// the tiles' sums, and puts its sum into every CTA's shared memory, with one cluster barrier.
// The last token's CTA is found from the CTAs' sums, its tile from the tiles' sums, and only
// that tile is read again.
//
// What bounds it.  One request (8 drafts, 32000 tokens) takes 8.3 us: 2 until the tree and its
// probabilities are there (two round trips), 1 for the walk, 1.2 for the sum, 1 for the barrier,
// then the draw.  128 requests x 5 drafts of 100003 tokens (102 MB, each row pair summed once) take
// 25.5 us, 59 % of the copy rate: the sums themselves 12, in which every request starts and ends
// at about the same time.  64 x 8 drafts of 131072 tokens take 39 us, as long as the request with
// the most children that fall: 7 us for the first sum of all, 6 for every further one of a few
// (4 of them reading from L1 and L2, the loads of 8 warps an SM in flight; through shared memory,
// four pieces of 1 KB a warp ahead, the call takes 56 us: L1 has then no room for the rows).
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
// All CTAs of a call are on the GPU at once, if the requests are few enough, with as many a request
// as that leaves.  128 x 5 drafts of 100003 tokens: 4 CTAs an SM 25.5 us (4 a request), 5 (48 registers)
// 33.2; and, measured when the first of these took 27.8: 3 an SM 29.8, 2 a request 31.4, 8 (in two
// rounds) 33.1, 16 53.5.  64 x 8 of 131072 then: 8 a request 40.7, 4 53.6, 16 43.5.
constexpr int kCtasPerSm = 4;
// Values of each row that a lane reads at once (8: 64 x 8 drafts 42.7 us instead of 39.8, one request
// 7.8 instead of 8.3).
constexpr int kPerLane = 16;
constexpr int kSpan = 32 * kPerLane;
constexpr int kMaxTiles = 256;

using u64 = unsigned long long;
constexpr u64 kOne = 1ull << 62;   // 1 as a multiple of 2^-62 (probabilities, W)
constexpr u64 kUnit = 1ull << 54;  // 1 as a multiple of 2^-54 (A: 1 + 254 W below 4 at most, 1017)
constexpr int kToUnit = 8;         // bits between the two (W and A are multiples of 2^-44: none is lost)

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
// a b 2^-62, rounded down.
__device__ __forceinline__ u64 share_of(u64 a, u64 b) { return (__umul64hi(a, b) << 2) | ((a * b) >> 62); }
// Whether a b 2^-62 < c, exactly.
__device__ __forceinline__ bool product_below(u64 a, u64 b, u64 c) {
  const u64 hi = __umul64hi(a, b), lo = a * b;
  return hi < c >> 2 || (hi == c >> 2 && lo < c << 62);
}
// max(p - A q, 0) of one token, A q rounded down to a multiple of 2^-62 (so that nothing is left
// where A q is p or more).
__device__ __forceinline__ u64 left(float p, float q, u64 A) {
  if (product(q, A) >= 2 * kUnit) return 0;
  const uint32_t bits = __float_as_uint(__saturatef(q));
  const uint32_t m = (bits << 8) | 0x80000000u, e = bits >> 23;  // q = m 2^(e - 158)
  const u64 w = fixed(p);
  const u64 off = e < 55u ? 0 : static_cast<u64>((static_cast<unsigned __int128>(A) * m) >> (150u - e));
  return off >= w ? 0 : w - off;
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
__device__ __forceinline__ void store_remote(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}

// The sums' form of values in [0, 1]: hi 2^-22 + lo 2^-44 (added up modulo 2^32, with an offset
// for each value).
struct Halves {
  uint32_t hi, lo;
};
constexpr uint32_t kHiOffset = 0x40000000u, kLoOffset = 0x35400000u;  // 2, 1.5 x 2^-21
__device__ __forceinline__ u64 whole(Halves h, uint32_t n) {  // of n values, as a multiple of 2^-62
  const long long hi = h.hi - n * kHiOffset;                  // (2^22 n at most: n below 1024)
  const int lo = static_cast<int>(h.lo - n * kLoOffset);      // (1.25 x 2^21 n at most: n up to 512)
  return static_cast<u64>((hi << 22) + lo) << 18;
}
// Of d + e for a pair of values, |e| at most 2^-25.
__device__ __forceinline__ void halves(float2 d, float2 e, Halves& x, Halves& y) {
  const float2 t = __fadd2_rn(d, make_float2(2.f, 2.f));
  const float2 back = __fadd2_rn(t, make_float2(-2.f, -2.f));
  const float2 r = __fadd2_rn(d, make_float2(-back.x, -back.y));  // exact, 2^-23 at most
  const float2 u = __fadd2_rn(__fadd2_rn(r, e), make_float2(0x1.8p-21f, 0x1.8p-21f));
  x = Halves{__float_as_uint(t.x), __float_as_uint(u.x)};
  y = Halves{__float_as_uint(t.y), __float_as_uint(u.y)};
}
// Of max(p - A q, 0), A as the sum of two fp32 (hi, lo): A q = t + l with l = the product's
// rounding error + lo q, and p - t = d + an error that is computed exactly.  Whether something is
// left, and what, is up to the sum s of d and e: where the product rounds to p or past it, d alone
// is 0 or negative.  (s, d - s + e) is the same sum with a second part of 2^-25 at most, as s is 1 at
// most.  Where s is positive t is below 1 + 2^-22, so that |l| is little more than 2^-23 at most, and
// what is lost is 2^-48 of A q in A's two parts, 2^-47 in l and e, 2^-48 in the second part, and 2^-47
// in halves before its rounding to 2^-44.
template <bool FALLEN>
__device__ __forceinline__ void left_halves(float2 p, float2 q, float2 A, Halves& x, Halves& y) {
  p = make_float2(__saturatef(p.x), __saturatef(p.y));
  if constexpr (!FALLEN) {
    halves(p, make_float2(0.f, 0.f), x, y);
  } else {
    q = make_float2(-__saturatef(q.x), -__saturatef(q.y));
    const float2 h = make_float2(A.x, A.x), lo = make_float2(A.y, A.y);
    const float2 t = __fmul2_rn(q, h);
    const float2 l = __ffma2_rn(q, lo, __ffma2_rn(q, h, make_float2(-t.x, -t.y)));
    const float2 d = __fadd2_rn(p, t);
    float2 e = __fadd2_rn(__fadd2_rn(__fadd2_rn(p, make_float2(-d.x, -d.y)), t), l);
    const float2 s = __fadd2_rn(d, e);
    const float2 rest = __fadd2_rn(__fadd2_rn(d, make_float2(-s.x, -s.y)), e);
    const bool x_left = s.x > 0.f, y_left = s.y > 0.f;
    halves(make_float2(x_left ? s.x : 0.f, y_left ? s.y : 0.f),
           make_float2(x_left ? rest.x : 0.f, y_left ? rest.y : 0.f), x, y);
  }
}
// The same of one token.
__device__ __forceinline__ u64 left_rounded(float p, float q, float2 A, bool fallen) {
  Halves x, y;
  if (fallen)
    left_halves<true>(make_float2(p, 0.f), make_float2(q, 0.f), A, x, y);
  else
    left_halves<false>(make_float2(p, 0.f), make_float2(0.f, 0.f), A, x, y);
  return whole(x, 1);
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

// The sum over a span of tokens, found by a warp together.
template <typename T, bool FALLEN>
__device__ __forceinline__ u64 span_sum(const T* pr, const T* qr, int b, int end, float2 A) {
  const int i = b + (threadIdx.x & 31);
  const bool all = b + kSpan <= end;
  float a[kPerLane], d[kPerLane];
  read_span(pr, i, end, all, a);
  if (FALLEN) read_span(qr, i, end, all, d);
  Halves s{0, 0};
#pragma unroll
  for (int k = 0; k < kPerLane; k += 2) {
    Halves x, y;
    left_halves<FALLEN>(make_float2(a[k], a[k + 1]),
                        FALLEN ? make_float2(d[k], d[k + 1]) : make_float2(0.f, 0.f), A, x, y);
    s.hi += x.hi + y.hi;
    s.lo += x.lo + y.lo;
  }
  static_assert(kSpan <= 512, "sums of a span's values in 32 bits");
  s.hi = __reduce_add_sync(0xffffffffu, s.hi);
  s.lo = __reduce_add_sync(0xffffffffu, s.lo);
  return whole(s, kSpan);
}

// What a walk decides: the sums of max(p - A q, 0) at a node, or the draw.
enum : int { kDone, kSum, kDraw };
struct Step {
  int op, node;
  u64 A;  // kDraw: where the random number falls in the running sum
};

template <typename T, bool DRAWN>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) draft_verify_kernel(const VerifyParams p) {
  __shared__ int parent[kMaxNodes], token[kMaxNodes], path[kMaxNodes];
  __shared__ u64 chance[kMaxNodes];            // u, p and q of every node
  __shared__ float pv[kMaxNodes], qv[kMaxNodes];
  __shared__ u64 sums[kMaxTiles];              // of this CTA's tiles
  __shared__ u64 totals[2][kMaxCtas];          // of all CTAs, of the last two sums
  __shared__ u64 part[kWarps];
  __shared__ int nodes;
  __shared__ Step step;
  // A and W of the walk, kept here as the sums need the registers (128 x 5 drafts 27.8 us -> 25.5)
  __shared__ u64 walk[2];
  __shared__ int gone[DRAWN ? 1 : kMaxNodes];  // without a draft: tokens that have fallen at the node
  const int ctas = cluster_size(), rank = cluster_rank();
  const int r = blockIdx.x / ctas;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  const T* p_rows = static_cast<const T*>(p.p) + r * p.p_stride[0];
  const T* q_rows = DRAWN ? static_cast<const T*>(p.q) + r * p.q_stride[0] : nullptr;
  if (tid == 0) {
    walk[0] = 0;
    walk[1] = kOne;
  }
  cluster_arrive();  // (shared memory of another CTA may be written once it has started)
  if (rank == 0) {
    const size_t row = static_cast<size_t>(r) * p.Tn;
    int n = p.Tn, up = -1, x = -1;
    float u = 0.f, a = 0.f, b = DRAWN ? 0.f : 1.f;
    if (p.tree_lens) n = p.tree_lens[r];
    if (tid < p.Tn) {
      up = p.parents[row + tid];
      x = p.tokens[row + tid];
      u = p.uniforms[row + tid];
    }
    const bool bad_n = n < 0 || n > p.Tn;
    const bool bad = !bad_n && tid < n && (up < -1 || up >= tid);
    if (!bad_n && !bad && tid < n && up >= 0 && x >= 0 && x < p.V) {
      a = value(p_rows[up * p.p_stride[1] + x]);
      if (DRAWN) b = value(q_rows[up * p.q_stride[1] + x]);
    }
    const bool bad_tree = __syncthreads_or(bad);
    if ((bad_n || bad_tree) && tid == 0) raise_flag(p.flags, bad_n ? DEVFLAG_BAD_SEQLEN : DEVFLAG_BAD_TREE);
    if (bad_n || bad_tree) n = 0;
    if (tid == 0) path[0] = 0;
    cluster_wait();
    for (int c = 0; c < ctas; ++c) {
      if (tid == 0) store_remote(remote(&nodes, c), static_cast<uint32_t>(n));
      if (tid >= n) continue;
      store_remote(remote(&parent[tid], c), static_cast<uint32_t>(up));
      store_remote(remote(&token[tid], c), static_cast<uint32_t>(x));
      store_remote(remote(&chance[tid], c), fixed(u));
      store_remote(remote(&pv[tid], c), __float_as_uint(a));
      store_remote(remote(&qv[tid], c), __float_as_uint(b));
    }
  } else {
    cluster_wait();
  }
  cluster_arrive();
  cluster_wait();
  const int n = nodes;

  // the walk (warp 0)
  int cur = 0, at = 0, fallen = 0, count = n > 0 ? 1 : 0;
  enum { kNothing, kAfterFall, kFalls, kLast } waiting = kNothing;
  bool summed = false;  // the last sums are those of the present w
  int buffer = 0;       // of totals that the next sums go to
  Step now{kDone, 0, 0};
  float2 A2 = make_float2(0.f, 0.f);
  const int c0 = rank * p.chunk, c1 = min(p.V, c0 + p.chunk);  // (chunk * ctas < 2^31)
  auto fallen_already = [&](int x) {
    bool hit = false;
    for (int i = lane; i < fallen; i += 32) hit |= gone[i] == x;
    return __any_sync(0xffffffffu, hit) != 0;
  };

  for (;;) {
    if (warp == 0) {
      u64 A = walk[0], W = walk[1];
      Step next{kDone, cur, 0};
      u64 all = 0;  // the sum over the row as it is now (once there is one)
      bool again = waiting == kFalls;  // child `at` is known to fall
      if (waiting != kNothing) {
        all = warp_sum(lane < ctas ? totals[buffer ^ 1][lane] : 0);
        summed = waiting != kAfterFall || all > 0;
        if (waiting == kAfterFall && all > 0) {
          A += W >> kToUnit;
          W = all;
        }
      }
      waiting = kNothing;
      while (n > 0) {
        if (!again) {
          // the next child of the node reached
          int found = -1;
          for (int b = (at + 1) & ~31; b < n && found < 0; b += 32) {
            const int i = b + lane;
            const unsigned hit = __ballot_sync(0xffffffffu, i > at && i < n && parent[i] == cur);
            if (hit) found = b + __ffs(hit) - 1;
          }
          if (found < 0) {
            next.op = summed ? kDraw : kSum;
            next.A = A;
            waiting = kLast;
            break;
          }
          at = found;
          u64 w;
          if (DRAWN) {
            w = A == 0 ? fixed(pv[at]) : left(pv[at], qv[at], A);
          } else {
            w = fallen_already(token[at]) ? 0 : fixed(pv[at]);
          }
          if (product_below(chance[at], DRAWN ? product(qv[at], W) : W, w)) {
            if (lane == 0) path[count] = at;
            ++count;
            cur = next.node = at;
            fallen = 0;
            A = 0;
            W = kOne;
            summed = false;
            continue;
          }
        }
        again = false;
        if (DRAWN) {
          next.op = kSum;
          next.A = A + (W >> kToUnit);
          waiting = kAfterFall;
          break;
        }
        if (!summed) {
          next.op = kSum;
          waiting = kFalls;
          break;
        }
        // without a draft it is the token itself that falls: it leaves the sums, and is gone for
        // the node's other children even where it is too small for the sums
        const int x = token[at];
        const float px = fallen_already(x) ? 0.f : pv[at];
        const u64 w = left_rounded(px, 0.f, A2, false);
        if (all > w) {
          all -= w;
          W = all;
          if (px > 0.f) {  // (x is one of the V)
            if (lane == 0) {
              gone[fallen] = x;
              const int c = x / p.chunk;
              totals[buffer ^ 1][c] -= w;
              if (c == rank) sums[(x - c0) / p.tile] -= w;
            }
            ++fallen;
            __syncwarp();
          }
        }
      }
      if (next.op == kDraw) {
        next.A = share_of(chance[0], all);
        if (all == 0) {
          next.op = kDone;
          if (rank == 0 && lane == 0) raise_flag(p.flags, DEVFLAG_NO_MASS);
        }
      }
      __syncwarp();
      if (lane == 0) {
        step = next;
        walk[0] = A;
        walk[1] = W;
      }
    }
    __syncthreads();
    if (step.op != kSum) break;

    // ---- sums of this CTA's tokens ----
    now = step;
    A2.x = __ull2float_rn(now.A) * 0x1p-54f;
    // (both are below 2^64, and their difference is small)
    A2.y = __ll2float_rn(static_cast<long long>(now.A - __float2ull_rn(A2.x * 0x1p54f))) * 0x1p-54f;
    const T* pr = p_rows + now.node * p.p_stride[1];
    const T* qr = DRAWN ? q_rows + now.node * p.q_stride[1] : nullptr;
    u64 mine = 0;
    for (int t = warp; c0 + t * p.tile < c1; t += kWarps) {
      u64 sum = 0;
      const int end = min(c1, c0 + (t + 1) * p.tile);
      for (int b = c0 + t * p.tile; b < end; b += kSpan)
        sum += DRAWN && now.A != 0 ? span_sum<T, DRAWN>(pr, qr, b, end, A2)
                                   : span_sum<T, false>(pr, qr, b, end, A2);
      if (lane == 0) sums[t] = sum;
      mine += sum;
    }
    if (lane == 0) part[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      mine = warp_sum(lane < kWarps ? part[lane] : 0);
      if (lane < ctas) store_remote(remote(&totals[buffer][rank], lane), mine);
    }
    // (a CTA writes a buffer again two sums on: every other one has then read it)
    buffer ^= 1;
    cluster_arrive();
    cluster_wait();
  }

  // ---- results ----
  const Step last = step;
  const size_t row = static_cast<size_t>(r) * p.Tn;
  if (warp != 0) return;
  if (rank == 0) {
    for (int j = lane; j < p.Tn; j += 32) {
      p.path[row + j] = j < count ? path[j] : -1;
      if (last.op == kDone || j != count - 1)  // (the last token is written by its CTA)
        p.tokens_out[row + j] = j < count - 1 ? token[path[j + 1]] : -1;
    }
    if (lane == 0) p.counts[r] = count;
  }
  if (last.op != kDraw) return;
  // the CTA whose tokens the running sum passes the drawn place in (the first one writes that
  // there is none, which sums past 64 bits can lead to)
  const int n_gone = DRAWN ? 0 : fallen;
  const u64 own = lane < ctas ? totals[buffer ^ 1][lane] : 0;
  const u64 upto = warp_prefix(own);
  const unsigned passes = __ballot_sync(0xffffffffu, last.A - (upto - own) < own);
  if (rank != max(__ffs(passes), 1) - 1) return;  // (1: CTA 0)
  u64 rest = last.A - __shfl_sync(0xffffffffu, upto - own, rank);
  // its tile
  const int tiles = (c1 - c0 + p.tile - 1) / p.tile;
  int t = -1;
  for (int b = 0; passes != 0 && b < tiles && t < 0; b += 32) {
    const u64 s = b + lane < tiles ? sums[b + lane] : 0;
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
  const T* pr = p_rows + now.node * p.p_stride[1];
  const T* qr = DRAWN ? q_rows + now.node * p.q_stride[1] : nullptr;
  const bool subtract = DRAWN && now.A != 0;
  const int end = min(c1, c0 + (t + 1) * p.tile);
  for (int b = c0 + t * p.tile; t >= 0 && b < end; b += kSpan) {
    const int i0 = b + kPerLane * lane;
    unsigned out = 0;  // values that have fallen
    for (int i = 0; i < n_gone; ++i) {
      const unsigned x = static_cast<unsigned>(gone[i] - i0);
      if (x < kPerLane) out |= 1u << x;
    }
    u64 w[kPerLane], sum = 0;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      w[k] = 0;
      if (i0 + k < end && !(out >> k & 1u))
        w[k] = left_rounded(value(pr[i0 + k]), subtract ? value(qr[i0 + k]) : 0.f, A2, subtract);
      sum += w[k];
    }
    const u64 incl = warp_prefix(sum);
    const unsigned hit = __ballot_sync(0xffffffffu, rest < incl);
    if (hit) {
      if (lane == __ffs(hit) - 1) {
        u64 s = incl - sum;
        int x = i0;
#pragma unroll
        for (int k = 0; k < kPerLane; ++k) {  // (as many values as leave the sum at `rest` or below)
          s += w[k];
          if (s <= rest) x = i0 + k + 1;
        }
        p.tokens_out[row + count - 1] = x;
      }
      return;
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) {
    p.tokens_out[row + count - 1] = -1;
    raise_flag(p.flags, DEVFLAG_NO_MASS);
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
  while (ctas > 1 && static_cast<long long>(p.S) * ctas > kCtasPerSm * num_sms) ctas /= 2;
  while (ctas > 1 && p.V <= ctas / 2 * kSpan * kWarps) ctas /= 2;
  auto up = [](long long x, long long m) { return (x + m - 1) / m * m; };
  const long long share = (static_cast<long long>(p.V) + ctas - 1) / ctas;
  p.tile = static_cast<int>(up((share + kMaxTiles - 1) / kMaxTiles, kSpan));
  p.chunk = static_cast<int>(up(share, p.tile));
  if (bf16)
    return p.q ? launch<uint16_t, true>(p, ctas, stream) : launch<uint16_t, false>(p, ctas, stream);
  return p.q ? launch<float, true>(p, ctas, stream) : launch<float, false>(p, ctas, stream);
}

}  // namespace gbattn
