// kv_keep.cu -- keeping chosen rows behind a request's cache and moving them together:
// what is left to do in the paged cache once it is known which drafted tokens stand.
//
// For every layer, K or V, and KV head, row L + path[j] goes to row L + j, j < count.  The
// path increases, so a row is never written before it has been read if the rows go in
// order, and rows are cut into 16-byte columns that one lane each moves from row to row:
// no lane reads what another one writes, and a lane reads several rows ahead of its
// stores.
//
// Pure data movement, 4 D bytes a row read and as many written.  A CTA translates the rows
// of a request through the block table once and moves them for some of the request's
// (layer, K or V, KV head) items.  The time is that of a chain of five round trips (lengths, path,
// table, row in, row out): one layer of 4 requests 3.2 us, 32 layers of 64 requests (13 MB, 2 us at
// the copy rate) 6.4, with 8 rows ahead 7.2 (fewer warps fit), with 4 CTAs an SM 9.4.
#include <cuda_runtime.h>

#include "gbattn.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "tree.h"

namespace gbattn {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // rows a lane reads before it stores them

template <int D>
__global__ void __launch_bounds__(kThreads) paged_kv_keep_kernel(const __grid_constant__ KeepParams p) {
  constexpr int CH = D / 8;  // 16-byte columns of a row
  __shared__ int from[GBATTN_TREE_MAX_NODES], to[GBATTN_TREE_MAX_NODES];
  const int r = blockIdx.x;
  // an attention launched next as a programmatic dependent may set itself up; it waits for
  // this grid's writes before it reads anything
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int L = p.seq_lens[r], n = p.counts[r];
  const int j = threadIdx.x;
  static_assert(kThreads == GBATTN_TREE_MAX_NODES, "a thread a row");
  const bool sizes_ok = L >= 0 && n >= 0 && n <= p.path_len;
  const bool mine = sizes_ok && j < n;
  const int32_t* path = p.path + static_cast<size_t>(r) * p.path_len;
  const int at = mine ? path[j] : 0;
  const int before = mine && j > 0 ? path[j - 1] : -1;
  const bool increases = !mine || (at > before && at >= j);
  const bool fits = sizes_ok && static_cast<long long>(L) + (mine ? at : 0) <
                                    static_cast<long long>(p.max_blocks) * kPagedBlock + (mine ? 0 : 1);
  const bool bad_path = __syncthreads_or(!increases);
  const bool bad_size = __syncthreads_or(!fits);
  if (bad_path || bad_size) {
    if (blockIdx.y == 0 && j == 0) {
      raise_flag(p.flags, bad_size ? DEVFLAG_BAD_SEQLEN : DEVFLAG_BAD_TREE);
      if (p.new_seq_lens) p.new_seq_lens[r] = L;
    }
    return;
  }
  if (blockIdx.y == 0 && j == 0 && p.new_seq_lens) p.new_seq_lens[r] = L + n;
  // rows 0 .. first - 1 stay in place
  const int first = __syncthreads_count(mine && at == j);
  if (mine && j >= first) {
    // first row of a KV head 0 of the block, and the slot; -1: a block outside the pool
    const int s = L + at, d = L + j;
    int a = paged_block_row(p.block_table, p.max_blocks, r, s / kPagedBlock, 0, p.Hkv,
                            p.num_pool_blocks);
    const int b = paged_block_row(p.block_table, p.max_blocks, r, d / kPagedBlock, 0, p.Hkv,
                                  p.num_pool_blocks);
    if (a < 0 || b < 0) {
      if (blockIdx.y == 0) raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
      a = -1;
    }
    from[j] = a < 0 ? -1 : a + s % kPagedBlock;
    to[j] = b + d % kPagedBlock;
  }
  __syncthreads();
  if (first >= n) return;

  const int lane = threadIdx.x % CH;  // column
  const int items = 2 * p.layers * p.Hkv;
  const int step = gridDim.y * (kThreads / CH);
  for (int i = blockIdx.y * (kThreads / CH) + threadIdx.x / CH; i < items; i += step) {
    const int h = i % p.Hkv, kv = i / p.Hkv;
    uint4* rows = static_cast<uint4*>(p.pool[kv & 1][kv >> 1]) +
                  static_cast<size_t>(h) * (kPagedBlock * CH) + lane;
    for (int j0 = first; j0 < n; j0 += kAhead) {
      uint4 x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (j0 + k < n && from[j0 + k] >= 0) x[k] = rows[static_cast<size_t>(from[j0 + k]) * CH];
#pragma unroll
      for (int k = 0; k < kAhead; ++k)
        if (j0 + k < n && from[j0 + k] >= 0) rows[static_cast<size_t>(to[j0 + k]) * CH] = x[k];
    }
  }
}

}  // namespace

cudaError_t launch_kv_keep(const KeepParams& p, int D, int num_sms, cudaStream_t stream) {
  if (p.S <= 0 || p.layers <= 0) return cudaSuccess;
  const int per_cta = kThreads / (D / 8);
  const long long sets = (2ll * p.layers * p.Hkv + per_cta - 1) / per_cta;
  // some 16 CTAs an SM in all
  const long long want = (16ll * num_sms + p.S - 1) / p.S;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.S), static_cast<unsigned>(sets < want ? sets : want));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, D == 64 ? paged_kv_keep_kernel<64> : paged_kv_keep_kernel<128>, p);
}

}  // namespace gbattn
