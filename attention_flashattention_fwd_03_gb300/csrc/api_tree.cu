// api_tree.cu -- C entry points of the operators for trees of drafted tokens
// (include/gbattn.h): argument checks and launches, under the rules of api.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <new>

#include "api.h"
#include "gbattn.h"
#include "tree.h"

using namespace gbattn;

namespace {

constexpr int64_t kMaxStride = 1ll << 48;

bool good_strides(const int64_t* s) {
  return s && s[0] >= 0 && s[0] <= kMaxStride && s[1] >= 0 && s[1] <= kMaxStride;
}

bool overlap(const void* a, size_t a_bytes, const void* b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Whether two of the pools share memory.  A model's pools, one after another in one tensor or
// allocated in turn, are often in order: those need no copy.
bool pools_overlap(void* const* k, void* const* v, int n, size_t bytes, bool* out_of_memory) {
  auto apart = [&](uintptr_t a, uintptr_t b) { return a + bytes <= b; };
  auto at = [](void* p) { return reinterpret_cast<uintptr_t>(p); };
  auto ordered = [&](void* const* x) {
    for (int i = 1; i < n; ++i)
      if (!apart(at(x[i - 1]), at(x[i]))) return false;
    return true;
  };
  if (ordered(k) && ordered(v) && (apart(at(k[n - 1]), at(v[0])) || apart(at(v[n - 1]), at(k[0]))))
    return false;
  uintptr_t small[256];
  uintptr_t* all = 2ll * n <= 256 ? small : new (std::nothrow) uintptr_t[2 * static_cast<size_t>(n)];
  *out_of_memory = all == nullptr;
  if (!all) return false;
  for (int i = 0; i < n; ++i) {
    all[i] = at(k[i]);
    all[n + i] = at(v[i]);
  }
  std::sort(all, all + 2 * static_cast<size_t>(n));
  bool overlap = false;
  for (size_t i = 1; i < 2 * static_cast<size_t>(n); ++i) overlap |= !apart(all[i - 1], all[i]);
  if (all != small) delete[] all;
  return overlap;
}

// Whether the kernels' 32-bit counts hold a call of these sizes: query rows, and steps of
// 128 keys of every segment, 20 units each and 20 more a segment.
bool tree_fits(int S, int Tn, int Hq, int Hkv, int max_seq_len) {
  const unsigned __int128 rows = static_cast<unsigned __int128>(S) * Hq * Tn;
  const uint64_t tiles = (static_cast<uint64_t>(max_seq_len) + 127) / 128 + 1;
  const unsigned __int128 segs = static_cast<unsigned __int128>(S) * Hkv * tree_rounds(Hq / Hkv, Tn);
  return rows < kMaxDim && segs * (tiles + 1) * 20 < kMaxDim;
}

}  // namespace

GBATTN_API size_t paged_attn_tree_workspace_size(int num_seqs, int Tn, int Hq, int Hkv, int D,
                                                 int max_seq_len) {
  if (num_seqs <= 0 || Tn <= 0 || Tn > GBATTN_TREE_MAX_NODES || Hq <= 0 || Hkv <= 0 ||
      Hq % Hkv != 0 || Hq / Hkv > 128 || (D != 64 && D != 128) || max_seq_len < 0 ||
      !tree_fits(num_seqs, Tn, Hq, Hkv, max_seq_len))
    return 0;
  return tree_attn_workspace_bytes(num_seqs, Tn, Hq, Hkv, D, max_seq_len);
}

GBATTN_API int paged_attn_tree(const void* q, const void* k_pool, const void* v_pool,
                               const int32_t* block_table, const int32_t* seq_lens,
                               const int32_t* parents, const int32_t* tree_lens, int block_size,
                               int num_seqs, int Tn, int Hq, int Hkv, int D,
                               int max_blocks_per_seq, int num_pool_blocks, int max_seq_len,
                               float scale, void* o, float* lse, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (num_seqs < 0 || Tn < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq <= 0 ||
      num_pool_blocks <= 0 || max_seq_len < 0)
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (block_size != 16 || (D != 64 && D != 128) || Tn > GBATTN_TREE_MAX_NODES || Hq / Hkv > 128)
    return ATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0 || Tn == 0) return ATTN_OK;
  if (!q || !k_pool || !v_pool || !block_table || !seq_lens || !parents || !o)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_pool, 16) || !aligned(v_pool, 16) || !aligned(o, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(parents, 4) ||
      !aligned(tree_lens, 4) || !aligned(lse, 4))
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size >= kMaxDim ||
      static_cast<uint64_t>(max_blocks_per_seq) * block_size >= kMaxDim ||
      !tree_fits(num_seqs, Tn, Hq, Hkv, max_seq_len))
    return ATTN_ERR_UNSUPPORTED;
  const size_t need = tree_attn_workspace_bytes(num_seqs, Tn, Hq, Hkv, D, max_seq_len);
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* ds = nullptr;
  int st = device_state(&ds);
  if (st != ATTN_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  if ((st = encoder(&enc)) != ATTN_OK) return st;
  CUtensorMap tmQ, tmK, tmV;
  const uint64_t row_bytes = static_cast<uint64_t>(D) * 2;
  const uint32_t group = static_cast<uint32_t>(Hq / Hkv);
  const uint64_t q_strides[3] = {row_bytes * Tn, row_bytes, row_bytes * Tn * group};
  const uint64_t pool_strides[1] = {row_bytes};
  const uint32_t q_box[4] = {64, group, static_cast<uint32_t>(tree_tile_nodes(group, Tn)), 1};
  const uint32_t pool_box[2] = {64, 16};
  const uint64_t dq[4] = {static_cast<uint64_t>(D), group, static_cast<uint64_t>(Tn),
                          static_cast<uint64_t>(num_seqs) * Hkv};
  const uint64_t dpool[2] = {static_cast<uint64_t>(D),
                             static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size};
  if ((st = encode_bf16(enc, &tmQ, q, 4, dq, q_strides, q_box)) != ATTN_OK) return st;
  if ((st = encode_bf16(enc, &tmK, k_pool, 2, dpool, pool_strides, pool_box)) != ATTN_OK) return st;
  if ((st = encode_bf16(enc, &tmV, v_pool, 2, dpool, pool_strides, pool_box)) != ATTN_OK) return st;
  TreeParams p{};
  p.q = q;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.parents = parents;
  p.tree_lens = tree_lens;
  p.o = o;
  p.lse = lse;
  p.S = num_seqs;
  p.Tn = Tn;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.D = D;
  p.max_blocks = max_blocks_per_seq;
  p.num_pool_blocks = num_pool_blocks;
  p.max_seq_len = max_seq_len;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.flags = ds->flags;
  p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.withhold_copy = g_withhold_copy.load(std::memory_order_relaxed);
  return launch_tree_attn(tmQ, tmK, tmV, p, workspace, ds->num_sms,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

GBATTN_API int draft_verify(const void* target_probs, const void* draft_probs,
                            const int64_t* target_strides, const int64_t* draft_strides,
                            int prob_type, const int32_t* tokens, const int32_t* parents,
                            const float* uniforms, const int32_t* tree_lens, int num_seqs, int Tn,
                            int V, int32_t* tokens_out, int32_t* path, int32_t* counts,
                            void* stream) {
  if (num_seqs < 0 || Tn < 0 || V <= 0 || (prob_type != 0 && prob_type != 1))
    return ATTN_ERR_INVALID_ARG;
  // (a request's CTAs take 16 at most of a grid below 2^31)
  if (Tn > GBATTN_TREE_MAX_NODES || V >= (1 << 30) || num_seqs >= (1 << 26))
    return ATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0) return ATTN_OK;
  // (without nodes there are only counts to write)
  if (!counts || !good_strides(target_strides) || (draft_probs && !good_strides(draft_strides)) ||
      (Tn > 0 && (!target_probs || !tokens || !parents || !uniforms || !tokens_out || !path)))
    return ATTN_ERR_INVALID_ARG;
  const uintptr_t unit = prob_type == 0 ? 4 : 2;
  if (!aligned(target_probs, unit) || !aligned(draft_probs, unit) || !aligned(tokens, 4) ||
      !aligned(parents, 4) || !aligned(uniforms, 4) || !aligned(tree_lens, 4) ||
      !aligned(tokens_out, 4) || !aligned(path, 4) || !aligned(counts, 4))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* ds = nullptr;
  const int st = device_state(&ds);
  if (st != ATTN_OK) return st;
  VerifyParams p{};
  p.p = target_probs;
  p.q = draft_probs;
  for (int i = 0; i < 2; ++i) {
    p.p_stride[i] = target_strides[i];
    p.q_stride[i] = draft_probs ? draft_strides[i] : 0;
  }
  p.tokens = tokens;
  p.parents = parents;
  p.uniforms = uniforms;
  p.tree_lens = tree_lens;
  p.tokens_out = tokens_out;
  p.path = path;
  p.counts = counts;
  p.S = num_seqs;
  p.Tn = Tn;
  p.V = V;
  p.flags = ds->flags;
  return launch_draft_verify(p, prob_type == 1, ds->num_sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

GBATTN_API int paged_kv_keep(void* const* k_pools, void* const* v_pools, int num_layers,
                             const int32_t* block_table, const int32_t* seq_lens,
                             const int32_t* path, const int32_t* counts, int32_t* new_seq_lens,
                             int block_size, int num_seqs, int path_len, int Hkv, int D,
                             int max_blocks_per_seq, int num_pool_blocks, void* stream) {
  if (num_layers <= 0 || num_seqs < 0 || path_len < 0 || Hkv <= 0 || max_blocks_per_seq <= 0 ||
      num_pool_blocks <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (block_size != 16 || (D != 64 && D != 128) || path_len > GBATTN_TREE_MAX_NODES)
    return ATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0) return ATTN_OK;
  if (!k_pools || !v_pools || !block_table || !seq_lens || !counts || (!path && path_len > 0))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(path, 4) ||
      !aligned(counts, 4) || !aligned(new_seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  for (int i = 0; i < num_layers; ++i)
    if (!k_pools[i] || !v_pools[i] || !aligned(k_pools[i], 16) || !aligned(v_pools[i], 16))
      return ATTN_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size >= kMaxDim ||
      static_cast<uint64_t>(max_blocks_per_seq) * block_size >= kMaxDim)
    return ATTN_ERR_UNSUPPORTED;
  const size_t pool_bytes = static_cast<size_t>(num_pool_blocks) * Hkv * block_size * D * 2;
  bool out_of_memory = false;
  if (pools_overlap(k_pools, v_pools, num_layers, pool_bytes, &out_of_memory)) return ATTN_ERR_INVALID_ARG;
  if (out_of_memory) return ATTN_ERR_UNSUPPORTED;
  const size_t S = static_cast<size_t>(num_seqs);
  if (new_seq_lens &&
      (overlap(new_seq_lens, S * 4, seq_lens, S * 4) || overlap(new_seq_lens, S * 4, counts, S * 4) ||
       (path_len > 0 && overlap(new_seq_lens, S * 4, path, S * path_len * 4)) ||
       overlap(new_seq_lens, S * 4, block_table, S * max_blocks_per_seq * 4)))
    return ATTN_ERR_INVALID_ARG;
  DeviceState* ds = nullptr;
  const int st = device_state(&ds);
  if (st != ATTN_OK) return st;
  KeepParams p{};
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.path = path;
  p.counts = counts;
  p.S = num_seqs;
  p.path_len = path_len;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks_per_seq;
  p.num_pool_blocks = num_pool_blocks;
  p.flags = ds->flags;
  for (int l0 = 0; l0 < num_layers; l0 += kKeepLayers) {
    p.layers = num_layers - l0 < kKeepLayers ? num_layers - l0 : kKeepLayers;
    p.new_seq_lens = l0 == 0 ? new_seq_lens : nullptr;
    for (int i = 0; i < p.layers; ++i) {
      p.pool[0][i] = k_pools[l0 + i];
      p.pool[1][i] = v_pools[l0 + i];
    }
    if (launch_kv_keep(p, D, ds->num_sms, static_cast<cudaStream_t>(stream)) != cudaSuccess)
      return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}
