// tree.h -- launch interface of the operators for trees of drafted tokens: attention over
// the paged cache (tree_attn.cu), verification (draft_verify.cu) and keeping the accepted
// rows (kv_keep.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace gbattn {

constexpr int kTreeShortRows = 64;

struct TreeParams {
  const void* q;               // [S, Hq, Tn, D] bf16
  const int32_t* block_table;  // [S, max_blocks]
  const int32_t* seq_lens;     // [S]: tokens before the tree
  const int32_t* parents;      // [S, Tn]
  const int32_t* tree_lens;    // [S] or nullptr: Tn nodes everywhere
  void* o;                     // [S, Hq, Tn, D] bf16
  float* lse;                  // [S, Hq, Tn] or nullptr
  int S, Tn, Hq, Hkv, D;
  int max_blocks;
  int num_pool_blocks;
  int max_seq_len;
  float scale;
  float scale_log2;
  unsigned* flags;
  unsigned long long wait_limit_ns;
  int withhold_copy;           // test hook: the producer skips its first copy
};

size_t tree_attn_workspace_bytes(int S, int Tn, int Hq, int Hkv, int D, int max_seq_len);
cudaError_t prepare_tree_attn();
// tmQ is a 4-D map over [S * Hkv, group, Tn, D] with the group's heads next to the channels: a box
// of 64 channels x group heads x tree_tile_nodes(group, Tn) nodes x 1; tmK and tmV are the decode
// kernels' 2-D maps over the pools (64 x 16 box); all with the 128-byte swizzle.
int tree_tile_nodes(int group, int Tn);
// Segments of a KV head: how often a team of CTAs turns to it.
int tree_rounds(int group, int Tn);
cudaError_t launch_tree_attn(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                             const TreeParams& p, void* workspace, int num_sms,
                             cudaStream_t stream);

// The same for up to kTreeShortRows query rows on a KV head, without a workspace (tree_short.cu).
cudaError_t prepare_tree_short();
cudaError_t launch_tree_short(const CUtensorMap& tmK, const CUtensorMap& tmV, const TreeParams& p,
                              cudaStream_t stream);

struct VerifyParams {
  const void *p, *q;           // rows of V probabilities; q may be nullptr
  long long p_stride[2], q_stride[2];  // of requests and nodes, in elements
  const int32_t* tokens;       // [S, Tn]
  const int32_t* parents;      // [S, Tn]
  const float* uniforms;       // [S, Tn]
  const int32_t* tree_lens;    // [S] or nullptr
  int32_t *tokens_out, *path;  // [S, Tn]
  int32_t* counts;             // [S]
  int S, Tn, V;
  int chunk, tile;             // tokens of a CTA, and of a sum that it keeps (launcher)
  unsigned* flags;
};

cudaError_t prepare_draft_verify();
cudaError_t launch_draft_verify(VerifyParams p, bool bf16, int num_sms, cudaStream_t stream);

constexpr int kKeepLayers = 128;  // layers of one launch

struct KeepParams {
  void* pool[2][kKeepLayers];  // K and V pools of the layers
  const int32_t* block_table;  // [S, max_blocks]
  const int32_t* seq_lens;     // [S]
  const int32_t* path;         // [S, path_len]
  const int32_t* counts;       // [S]
  int32_t* new_seq_lens;       // [S] or nullptr
  int S, layers, path_len, Hkv;
  int max_blocks;
  int num_pool_blocks;
  unsigned* flags;
};

cudaError_t launch_kv_keep(const KeepParams& p, int D, int num_sms, cudaStream_t stream);

}  // namespace gbattn
