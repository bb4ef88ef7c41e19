// kv4_cache.cu -- reading a request's history out of the 4-bit paged cache.
//
// One CTA per (request, KV head, 16-token block), D / 8 lanes a token: a lane takes 8
// channels of the K row and of the V row, whose codes kv4.cuh places in one word and in
// two half words, multiplies by the group's scale (exact in bf16) and stores 16 bytes of
// each.  Memory-bound: 9 D / 8 bytes read and 4 D written a token and head.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "norm_rope.cuh"
#include "ptx.cuh"

namespace gbattn {

namespace {

template <int D>
__global__ void __launch_bounds__(2 * D) paged_kv4_gather_kernel(const Gather4Params p) {
  using F = Kv4<D>;
  constexpr int LANES = D / 8;
  const int n_blocks = (p.max_seq_len + kPagedBlock - 1) / kPagedBlock;
  const int lb = blockIdx.x % n_blocks;
  const int rh = blockIdx.x / n_blocks;
  const int h = rh % p.Hkv, r = rh / p.Hkv;
  const int L = p.seq_lens[r];
  if (L < 0 || L > p.max_seq_len || L > p.max_blocks * kPagedBlock) {
    if (threadIdx.x == 0 && lb == 0 && h == 0) raise_flag(p.flags, DEVFLAG_BAD_SEQLEN);
    return;
  }
  const int slot = threadIdx.x / LANES, l = threadIdx.x % LANES;
  const int t = lb * kPagedBlock + slot;
  if (t >= L) return;
  const long long phys = p.block_table[static_cast<size_t>(r) * p.max_blocks + lb];
  const bool bad = phys < 0 || phys >= p.num_pool_blocks;
  if (bad && threadIdx.x == 0) raise_flag(p.flags, DEVFLAG_BAD_BLOCK);
  uint4 k4, v4;
  k4 = v4 = make_uint4(kBf16NanPair, kBf16NanPair, kBf16NanPair, kBf16NanPair);
  if (!bad) {
    const uint8_t* chunk = p.pool + (phys * p.Hkv + h) * F::kChunk;
    const int group = l >> 2, part = l & 3;
    auto scale = [&](int off) {
      const uint16_t* s = reinterpret_cast<const uint16_t*>(chunk + off + slot * F::kScaleRow);
      return s[group] * 0x10001u;
    };
    const uint32_t kc = reinterpret_cast<const uint32_t*>(
        chunk + F::kOffKCodes + slot * F::kCodeRow)[part * F::kGroups + group];
    const uint16_t* vrow =
        reinterpret_cast<const uint16_t*>(chunk + F::kOffVCodes + slot * F::kCodeRow);
    const uint32_t vc = vrow[2 * part * F::kGroups + group] |
                        (static_cast<uint32_t>(vrow[(2 * part + 1) * F::kGroups + group]) << 16);
    k4 = kv4_values<64>(kc, scale(F::kOffKScales));
    v4 = kv4_values<64>(vc, scale(F::kOffVScales));
  }
  const size_t at = (static_cast<size_t>(rh) * p.max_seq_len + t) * D + 8 * l;
  *reinterpret_cast<uint4*>(p.k_out + at) = k4;
  *reinterpret_cast<uint4*>(p.v_out + at) = v4;
}

}  // namespace

cudaError_t launch_kv4_gather(const Gather4Params& p, int D, cudaStream_t stream) {
  const long long n_blocks = (p.max_seq_len + kPagedBlock - 1) / kPagedBlock;
  const long long grid = static_cast<long long>(p.S) * p.Hkv * n_blocks;
  if (grid <= 0) return cudaSuccess;
  if (D == 64)
    paged_kv4_gather_kernel<64><<<static_cast<unsigned>(grid), 128, 0, stream>>>(p);
  else
    paged_kv4_gather_kernel<128><<<static_cast<unsigned>(grid), 256, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gbattn
