// tree_attn.cu -- attention of the nodes of trees of drafted tokens over the paged cache.
#include <cuda_runtime.h>

#include "gbattn.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "tree.h"

namespace gbattn {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float bf16_value(uint16_t v) {
  return __uint_as_float(static_cast<uint32_t>(v) << 16);
}

// One CTA a (request, query head, node); its warps take the keys in turn.
template <int D>
__global__ void __launch_bounds__(kThreads) tree_attn_kernel(const TreeParams p) {
  constexpr int PER = D / 32;
  __shared__ unsigned seen[GBATTN_TREE_MAX_NODES / 32];
  __shared__ float part[kWarps][D], part_m[kWarps], part_l[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int node = blockIdx.x % p.Tn, rh = blockIdx.x / p.Tn;
  const int r = rh / p.Hq, kvh = (rh - r * p.Hq) / (p.Hq / p.Hkv);
  const int L = p.seq_lens[r], n = p.tree_lens ? p.tree_lens[r] : p.Tn;
  const int32_t* parents = p.parents + static_cast<size_t>(r) * p.Tn;
  const bool bad_len = L < 0 || n < 0 || n > p.Tn ||
                       static_cast<long long>(L) + n > p.max_seq_len ||
                       static_cast<long long>(L) + n > static_cast<long long>(p.max_blocks) * kPagedBlock;
  bool bad_node = false;
  for (int i = threadIdx.x; i < n && !bad_len; i += kThreads)
    bad_node |= parents[i] < -1 || parents[i] >= i;
  const bool bad_tree = __syncthreads_or(bad_node);
  const bool bad = bad_len || bad_tree;
  if (bad && threadIdx.x == 0) raise_flag(p.flags, bad_len ? DEVFLAG_BAD_SEQLEN : DEVFLAG_BAD_TREE);
  if (threadIdx.x < GBATTN_TREE_MAX_NODES / 32) seen[threadIdx.x] = 0;
  __syncthreads();
  const bool live = !bad && node < n;
  if (threadIdx.x == 0 && live)
    for (int a = node; a >= 0; a = parents[a]) seen[a >> 5] |= 1u << (a & 31);
  __syncthreads();

  const uint16_t* q = static_cast<const uint16_t*>(p.q) + static_cast<size_t>(blockIdx.x) * D + lane * PER;
  float x[PER], o[PER], m = -INFINITY, l = 0.f;
  for (int i = 0; i < PER; ++i) {
    x[i] = bf16_value(q[i]);
    o[i] = 0.f;
  }
  const int keys = live ? L + node + 1 : 0;
  for (int t = warp; t < keys; t += kWarps) {
    if (t >= L && !(seen[(t - L) >> 5] >> ((t - L) & 31) & 1)) continue;
    int row = paged_block_row(p.block_table, p.max_blocks, r, t / kPagedBlock, kvh, p.Hkv,
                              p.num_pool_blocks);
    if (row < 0) {
      if (lane == 0) raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
      row = kvh * kPagedBlock;
    }
    const size_t at = static_cast<size_t>(row + t % kPagedBlock) * D + lane * PER;
    const uint16_t* k = static_cast<const uint16_t*>(p.k_pool) + at;
    const uint16_t* v = static_cast<const uint16_t*>(p.v_pool) + at;
    float s = 0.f;
    for (int i = 0; i < PER; ++i) s = fmaf(x[i], bf16_value(k[i]), s);
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s);
    const float al = ex2((m - mn) * p.scale_log2), e = ex2((s - mn) * p.scale_log2);
    m = mn;
    l = l * al + e;
    for (int i = 0; i < PER; ++i) o[i] = o[i] * al + e * bf16_value(v[i]);
  }
  for (int i = 0; i < PER; ++i) part[warp][lane * PER + i] = o[i];
  if (lane == 0) {
    part_m[warp] = m;
    part_l[warp] = l;
  }
  __syncthreads();
  if (threadIdx.x >= D) return;
  float M = -INFINITY, tot = 0.f, out = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, part_m[w]);
  const float Ms = M == -INFINITY ? 0.f : M;
  for (int w = 0; w < kWarps; ++w) {
    const float f = ex2((part_m[w] - Ms) * p.scale_log2);
    tot = fmaf(f, part_l[w], tot);
    out = fmaf(f, part[w][threadIdx.x], out);
  }
  const float nan = __int_as_float(0x7fc00000);
  out = bad ? nan : (tot == 0.f ? 0.f : out / tot);
  static_cast<uint16_t*>(p.o)[static_cast<size_t>(blockIdx.x) * D + threadIdx.x] =
      static_cast<uint16_t>(pack_bf16x2(out, 0.f));
  if (p.lse != nullptr && threadIdx.x == 0)
    p.lse[blockIdx.x] = bad ? nan : Ms * p.scale + logf(tot);
}

}  // namespace

size_t tree_attn_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t prepare_tree_attn() { return cudaSuccess; }

cudaError_t launch_tree_attn(const TreeParams& p, int num_sms, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>(p.S) * p.Hq * p.Tn;
  if (p.D == 64)
    tree_attn_kernel<64><<<grid, kThreads, 0, stream>>>(p);
  else
    tree_attn_kernel<128><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gbattn
