// kv4_cache.cu -- reading a request's history out of the 4-bit paged cache.
//
// One CTA per (request, 16-token block, two KV heads), D / 8 lanes a token: a lane takes 8
// channels of the K row and of the V row, whose codes kv4.cuh places in one word and in
// two half words, multiplies by the group's scale (exact in bf16) and stores 16 bytes of
// each.  Memory-bound in kind: 9 D / 8 bytes read and 4 D written a token and head.  16
// requests of 512 tokens, 8 KV heads, D 128 (43 MB, 6.3 us at the copy rate): 10 us behind
// an append, with one head a CTA 11, four or eight 11.  No pipe is full (issue slots 57 %,
// ALU 43 %): the 2048 CTAs of two loads and four stores a lane come and go in 10 us.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "norm_rope.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

constexpr int kHeads = 2;  // KV heads of a CTA, their loads in flight together

template <int D>
__global__ void __launch_bounds__(2 * D) paged_kv4_gather_kernel(const Gather4Params p) {
  using F = Kv4<D>;
  constexpr int LANES = D / 8;
  const unsigned n_blocks = (p.max_seq_len + (kPagedBlock - 1u)) / kPagedBlock;
  const unsigned n_sets = (p.Hkv + kHeads - 1) / kHeads;
  const unsigned set = blockIdx.x % n_sets, rb = blockIdx.x / n_sets;
  const int lb = rb % n_blocks, r = rb / n_blocks;
  const int h0 = set * kHeads;
  // launched as a programmatic dependent: the preceding kernel's writes (an append's) are
  // complete and visible past this point
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // (both loads at once; an entry past the table's row is not read)
  const int L = p.seq_lens[r];
  const long long phys =
      lb < p.max_blocks ? p.block_table[static_cast<size_t>(r) * p.max_blocks + lb] : -1;
  if (L < 0 || L > p.max_seq_len || L > p.max_blocks * kPagedBlock) {
    if (threadIdx.x == 0 && lb == 0 && set == 0) raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
    return;
  }
  const int slot = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const int t = lb * kPagedBlock + slot;
  if (t >= L) return;
  const bool bad = phys < 0 || phys >= p.num_pool_blocks;
  if (bad && threadIdx.x == 0) raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
  const int group = l >> 2, part = l & 3;
  const uint8_t* chunk = p.pool + ((bad ? 0 : phys) * p.Hkv + h0) * F::kChunk;
  uint32_t kc[kHeads], vc[kHeads], ks[kHeads], vs[kHeads];
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (h0 + i >= p.Hkv) break;
    const uint8_t* c = chunk + i * F::kChunk;
    kc[i] = reinterpret_cast<const uint32_t*>(c + slot * F::kCodeRow)[part * F::kGroups + group];
    const uint16_t* v = reinterpret_cast<const uint16_t*>(c + F::kOffVCodes + slot * F::kCodeRow);
    vc[i] = v[2 * part * F::kGroups + group] |
            (static_cast<uint32_t>(v[(2 * part + 1) * F::kGroups + group]) << 16);
    ks[i] = reinterpret_cast<const uint16_t*>(c + F::kOffKScales + slot * F::kScaleRow)[group];
    vs[i] = reinterpret_cast<const uint16_t*>(c + F::kOffVScales + slot * F::kScaleRow)[group];
  }
#pragma unroll
  for (int i = 0; i < kHeads; ++i) {
    if (h0 + i >= p.Hkv) break;
    // a block that the table could not translate reads as NaN
    const uint32_t sk = bad ? kBf16NanPair : ks[i] * 0x10001u;
    const uint32_t sv = bad ? kBf16NanPair : vs[i] * 0x10001u;
    const size_t at =
        ((static_cast<size_t>(r) * p.Hkv + h0 + i) * p.max_seq_len + t) * D + 8 * l;
    *reinterpret_cast<uint4*>(p.k_out + at) = kv4_values<64>(kc[i], sk);
    *reinterpret_cast<uint4*>(p.v_out + at) = kv4_values<64>(vc[i], sv);
  }
}

}  // namespace

cudaError_t launch_kv4_gather(const Gather4Params& p, int D, cudaStream_t stream) {
  const long long n_blocks = (p.max_seq_len + (kPagedBlock - 1ll)) / kPagedBlock;
  const long long grid = static_cast<long long>(p.S) * ((p.Hkv + kHeads - 1) / kHeads) * n_blocks;
  if (grid <= 0) return cudaSuccess;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(2 * D);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, D == 64 ? paged_kv4_gather_kernel<64> : paged_kv4_gather_kernel<128>, p);
}

}  // namespace gbattn
