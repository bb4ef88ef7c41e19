// norm_rope.h -- launch interface of the norm + rotation kernels (norm_rope.cu) and of
// the cache appends built on the same pass.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace gbattn {

// One [B, T, H, D] bf16 operand with unit channel stride; strides in elements.
struct Heads {
  uint16_t* p;  // nullptr: absent
  long long sb, st, sh;
};

struct RopeParams {
  const uint16_t* q_weight;   // [D] bf16 or nullptr: queries are not normalised
  const uint16_t* k_weight;   // [D] bf16 or nullptr
  const float* cos_sin;       // [max_pos, rot], nullptr when rot == 0
  const int32_t* positions;   // [B, T] or nullptr: t (behind seq_lens[b] in the appends)
  float eps;
  int rot, max_pos, interleaved;
};

enum class RowSink { kContiguous, kPaged, kPaged4 };

struct NormRopeParams {
  Heads q, k, v;              // inputs; q absent: 0 query heads, v absent: 0 value heads
  RopeParams rope;
  int B, T, nq, nk, nv;       // nq, nk, nv: heads of each operand that the launch handles
  uint16_t* q_out;            // [B, nq, T, D]
  uint16_t *k_out, *v_out;    // kContiguous: [B, nk, T, D], [B, nv, T, D]
  // kPaged: the bf16 pools; kPaged4: the 4-bit pool
  uint16_t *k_pool, *v_pool;
  uint8_t* kv4_pool;
  const int32_t* block_table;  // [B, max_blocks]
  const int32_t* seq_lens;     // [B] lengths before the append
  int32_t* new_seq_lens;       // [B] or nullptr
  int max_blocks, num_pool_blocks;
  int chunks, rows_per_warp;   // a token's nq + nk + nv rows are cut into chunks (launcher)
  float one;                   // 1, which the compiler must not know (launcher)
  unsigned* flags;
};

cudaError_t prepare_norm_rope();  // per-device one-time attributes
cudaError_t launch_norm_rope(NormRopeParams p, int D, RowSink sink, int num_sms,
                             cudaStream_t stream);

struct NormRopeBwdParams {
  Heads q, k;                  // the forward's inputs (read only when there is a weight)
  const uint16_t *gq, *gk, *gv;  // gradients of the outputs, [B, H, T, D]
  Heads dq, dk, dv;            // gradients of the inputs, strided
  RopeParams rope;
  int B, T, nq, nk, nv;
  float* part;                 // [grid, 2, D] partial weight gradients (workspace)
  float *dwq, *dwk;            // [D] each
  unsigned* flags;
};

// CTAs of the backward kernel: a function of the sizes alone, so that the weight
// gradients are summed in the same order on every run.
int norm_rope_bwd_grid(int B, int T);
size_t norm_rope_bwd_workspace_bytes(int B, int T, int D);
cudaError_t launch_norm_rope_bwd(const NormRopeBwdParams& p, int D, cudaStream_t stream);

}  // namespace gbattn
