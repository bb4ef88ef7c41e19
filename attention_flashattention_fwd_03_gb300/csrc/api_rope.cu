// api_rope.cu -- C entry points of the norm + rotation pass, of the cache appends built
// on it, and of the 4-bit cache (include/gbattn.h): argument checks and launches, under
// the rules of api.cu.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "api.h"
#include "gbattn.h"
#include "internal.h"
#include "norm_rope.h"

using namespace gbattn;

namespace {

constexpr int64_t kMaxStride = 1ll << 48;

bool good_strides(const int64_t* s) {
  if (!s) return false;
  for (int i = 0; i < 3; ++i)
    if (s[i] < 0 || s[i] > kMaxStride || s[i] % 8 != 0) return false;
  return true;
}

// Whether a written [B, T, H, D] layout gives every element a place of its own: taken
// from the smallest stride up, each dimension steps past everything below it.
bool distinct_places(const int64_t* s, int B, int T, int H, int D) {
  struct Dim {
    int64_t stride, size;
  } d[3] = {{s[0], B}, {s[1], T}, {s[2], H}};
  std::sort(d, d + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
  __int128 extent = D;
  for (const Dim& x : d) {
    if (x.size <= 1) continue;
    if (x.stride < extent) return false;
    extent += static_cast<__int128>(x.stride) * (x.size - 1);
  }
  return true;
}

Heads heads(const void* p, const int64_t* s) {
  Heads h{};
  h.p = static_cast<uint16_t*>(const_cast<void*>(p));
  if (p) {
    h.sb = s[0];
    h.st = s[1];
    h.sh = s[2];
  }
  return h;
}

// Checks that need no sizes of the batch: ATTN_OK, or what is wrong.
int check_rope(const void* q_weight, const void* k_weight, const float* cos_sin,
               const int32_t* positions, int D, int rot_dim, int max_pos, int interleaved,
               float eps) {
  if (interleaved != 0 && interleaved != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || !(eps > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > D || (rot_dim > 0 && max_pos <= 0)) return ATTN_ERR_INVALID_ARG;
  if (rot_dim % 8 != 0) return ATTN_ERR_UNSUPPORTED;
  if ((rot_dim > 0) != (cos_sin != nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q_weight, 16) || !aligned(k_weight, 16) || !aligned(cos_sin, 16) ||
      !aligned(positions, 4))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

RopeParams rope_params(const void* q_weight, const void* k_weight, const float* cos_sin,
                       const int32_t* positions, int rot_dim, int max_pos, int interleaved,
                       float eps) {
  RopeParams r{};
  r.q_weight = static_cast<const uint16_t*>(q_weight);
  r.k_weight = static_cast<const uint16_t*>(k_weight);
  r.cos_sin = cos_sin;
  r.positions = positions;
  r.eps = eps;
  r.rot = rot_dim;
  r.max_pos = max_pos;
  r.interleaved = interleaved;
  return r;
}

// An input operand: present with good strides and a 16-byte aligned base.
bool good_input(const void* p, const int64_t* s) { return p && aligned(p, 16) && good_strides(s); }

// Sizes past the kernels' counts: 2^31 tokens or heads, or 2^32 rows (half a terabyte of
// them at D = 64), with which a launch stays below 2^31 CTAs: a CTA has at least four rows of
// its token.
bool too_many_rows(int B, int T, int Hq, int Hkv) {
  const unsigned __int128 n = static_cast<unsigned __int128>(B) * T;
  const uint64_t rows = static_cast<uint64_t>(Hq) + 2ull * Hkv;
  return n >= kMaxDim || rows >= kMaxDim || n * rows >= (1ull << 32);
}

bool overlap(const void* a, const void* b, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + bytes && y < x + bytes;
}

// The two appends: four = into the 4-bit pool (k_pool), else into the bf16 pools.
int append(bool four, const void* q, const void* k, const void* v, const int64_t* q_strides,
           const int64_t* k_strides, const int64_t* v_strides, const void* q_weight,
           const void* k_weight, const float* cos_sin, const int32_t* positions, void* k_pool,
           void* v_pool, const int32_t* block_table, const int32_t* seq_lens,
           int32_t* new_seq_lens, int block_size, int num_seqs, int Tn, int Hq, int Hkv, int D,
           int max_blocks_per_seq, int num_pool_blocks, int rot_dim, int max_pos, int interleaved,
           float eps, void* q_out, void* stream) {
  if (num_seqs < 0 || Tn < 0 || Hq < 0 || Hkv <= 0 || max_blocks_per_seq <= 0 ||
      num_pool_blocks <= 0)
    return ATTN_ERR_INVALID_ARG;
  if (block_size != 16 || (D != 64 && D != 128)) return ATTN_ERR_UNSUPPORTED;
  int st = check_rope(q_weight, k_weight, cos_sin, positions, D, rot_dim, max_pos, interleaved,
                      eps);
  if (st != ATTN_OK) return st;
  if (num_seqs == 0 || (Tn == 0 && !new_seq_lens)) return ATTN_OK;
  // the lengths are read by every CTA while one of them writes the new ones
  if (new_seq_lens && (!seq_lens || !aligned(seq_lens, 4) || !aligned(new_seq_lens, 4) ||
                       overlap(seq_lens, new_seq_lens, sizeof(int32_t) * num_seqs)))
    return ATTN_ERR_INVALID_ARG;
  if (Tn == 0)  // nothing to append: the lengths stay
    return cudaMemcpyAsync(new_seq_lens, seq_lens, sizeof(int32_t) * num_seqs,
                           cudaMemcpyDeviceToDevice, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? ATTN_OK
               : ATTN_ERR_CUDA;
  if ((q != nullptr) != (q_out != nullptr) || (q && Hq == 0)) return ATTN_ERR_INVALID_ARG;
  if (q && (!good_input(q, q_strides) || !aligned(q_out, 16))) return ATTN_ERR_INVALID_ARG;
  if (!good_input(k, k_strides) || !good_input(v, v_strides)) return ATTN_ERR_INVALID_ARG;
  if (!k_pool || !aligned(k_pool, 16) || (!four && (!v_pool || !aligned(v_pool, 16))) ||
      !block_table || !aligned(block_table, 4) || !seq_lens || !aligned(seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  if (too_many_rows(num_seqs, Tn, q ? Hq : 0, Hkv) ||
      static_cast<uint64_t>(max_blocks_per_seq) * block_size >= kMaxDim ||
      static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size >= kMaxDim)
    return ATTN_ERR_UNSUPPORTED;
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != ATTN_OK) return st;
  NormRopeParams p{};
  p.q = heads(q, q_strides);
  p.k = heads(k, k_strides);
  p.v = heads(v, v_strides);
  p.rope = rope_params(q_weight, k_weight, cos_sin, positions, rot_dim, max_pos, interleaved, eps);
  p.B = num_seqs;
  p.T = Tn;
  p.nq = q ? Hq : 0;
  p.nk = p.nv = Hkv;
  p.q_out = static_cast<uint16_t*>(q_out);
  if (four) {
    p.kv4_pool = static_cast<uint8_t*>(k_pool);
  } else {
    p.k_pool = static_cast<uint16_t*>(k_pool);
    p.v_pool = static_cast<uint16_t*>(v_pool);
  }
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.new_seq_lens = new_seq_lens;
  p.max_blocks = max_blocks_per_seq;
  p.num_pool_blocks = num_pool_blocks;
  p.flags = ds->flags;
  return launch_norm_rope(p, D, four ? RowSink::kPaged4 : RowSink::kPaged, ds->num_sms,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

}  // namespace

GBATTN_API int qkv_norm_rope(const void* q, const void* k, const void* v, const int64_t* q_strides,
                             const int64_t* k_strides, const int64_t* v_strides,
                             const void* q_weight, const void* k_weight, const float* cos_sin,
                             const int32_t* positions, int B, int T, int Hq, int Hkv, int D,
                             int rot_dim, int max_pos, int interleaved, float eps, void* q_out,
                             void* k_out, void* v_out, void* stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  int st = check_rope(q_weight, k_weight, cos_sin, positions, D, rot_dim, max_pos, interleaved,
                      eps);
  if (st != ATTN_OK) return st;
  if (B == 0 || T == 0) return ATTN_OK;
  const struct {
    const void* in;
    const int64_t* strides;
    const void* out;
    int n;
  } ops[3] = {{q, q_strides, q_out, Hq}, {k, k_strides, k_out, Hkv}, {v, v_strides, v_out, Hkv}};
  if (!q && !k && !v) return ATTN_ERR_INVALID_ARG;
  for (const auto& o : ops) {
    if ((o.in != nullptr) != (o.out != nullptr)) return ATTN_ERR_INVALID_ARG;
    if (o.in && (o.n == 0 || !good_input(o.in, o.strides) || !aligned(o.out, 16)))
      return ATTN_ERR_INVALID_ARG;
  }
  if (too_many_rows(B, T, Hq, Hkv)) return ATTN_ERR_UNSUPPORTED;
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != ATTN_OK) return st;
  NormRopeParams p{};
  p.q = heads(q, q_strides);
  p.k = heads(k, k_strides);
  p.v = heads(v, v_strides);
  p.rope = rope_params(q_weight, k_weight, cos_sin, positions, rot_dim, max_pos, interleaved, eps);
  p.B = B;
  p.T = T;
  p.nq = q ? Hq : 0;
  p.nk = k ? Hkv : 0;
  p.nv = v ? Hkv : 0;
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.flags = ds->flags;
  return launch_norm_rope(p, D, RowSink::kContiguous, ds->num_sms,
                          static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

GBATTN_API size_t qkv_norm_rope_bwd_workspace_size(int B, int T, int D) {
  if (B <= 0 || T <= 0 || D <= 0) return 0;
  return norm_rope_bwd_workspace_bytes(B, T, D);
}

GBATTN_API int qkv_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* dv_out,
                                 const void* q, const void* k, const int64_t* q_strides,
                                 const int64_t* k_strides, const void* q_weight,
                                 const void* k_weight, const float* cos_sin,
                                 const int32_t* positions, int B, int T, int Hq, int Hkv, int D,
                                 int rot_dim, int max_pos, int interleaved, float eps, void* dq,
                                 void* dk, void* dv, const int64_t* dq_strides,
                                 const int64_t* dk_strides, const int64_t* dv_strides,
                                 float* dq_weight, float* dk_weight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (B < 0 || T < 0 || Hq < 0 || Hkv < 0) return ATTN_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return ATTN_ERR_UNSUPPORTED;
  int st = check_rope(q_weight, k_weight, cos_sin, positions, D, rot_dim, max_pos, interleaved,
                      eps);
  if (st != ATTN_OK) return st;
  if ((q_weight != nullptr) != (dq_weight != nullptr) ||
      (k_weight != nullptr) != (dk_weight != nullptr) || !aligned(dq_weight, 4) ||
      !aligned(dk_weight, 4))
    return ATTN_ERR_INVALID_ARG;
  const bool empty = B == 0 || T == 0;
  const bool weights = q_weight || k_weight;
  if (empty && !weights) return ATTN_OK;
  if (!empty) {
    const struct {
      const void* g;
      const void* d;
      const int64_t* strides;
      int n;
    } ops[3] = {{dq_out, dq, dq_strides, Hq}, {dk_out, dk, dk_strides, Hkv},
                {dv_out, dv, dv_strides, Hkv}};
    if (!dq_out && !dk_out && !dv_out) return ATTN_ERR_INVALID_ARG;
    for (const auto& o : ops) {
      if ((o.g != nullptr) != (o.d != nullptr)) return ATTN_ERR_INVALID_ARG;
      if (!o.g) continue;
      if (o.n == 0 || !aligned(o.g, 16) || !good_input(o.d, o.strides) ||
          !distinct_places(o.strides, B, T, o.n, D))
        return ATTN_ERR_INVALID_ARG;
    }
    if (q_weight && (!dq_out || !good_input(q, q_strides))) return ATTN_ERR_INVALID_ARG;
    if (k_weight && (!dk_out || !good_input(k, k_strides))) return ATTN_ERR_INVALID_ARG;
    if (too_many_rows(B, T, Hq, Hkv)) return ATTN_ERR_UNSUPPORTED;
    if (weights && (!workspace || !aligned(workspace, 16) ||
                    workspace_bytes < norm_rope_bwd_workspace_bytes(B, T, D)))
      return ATTN_ERR_INVALID_ARG;
  }
  DeviceState* ds = nullptr;
  if ((st = device_state(&ds)) != ATTN_OK) return st;
  NormRopeBwdParams p{};
  if (!empty) {
    if (q_weight) p.q = heads(q, q_strides);
    if (k_weight) p.k = heads(k, k_strides);
    p.gq = static_cast<const uint16_t*>(dq_out);
    p.gk = static_cast<const uint16_t*>(dk_out);
    p.gv = static_cast<const uint16_t*>(dv_out);
    p.dq = heads(dq, dq_strides);
    p.dk = heads(dk, dk_strides);
    p.dv = heads(dv, dv_strides);
    p.nq = dq_out ? Hq : 0;
    p.nk = dk_out ? Hkv : 0;
    p.nv = dv_out ? Hkv : 0;
    p.part = weights ? static_cast<float*>(workspace) : nullptr;
  }
  p.rope = rope_params(q_weight, k_weight, cos_sin, positions, rot_dim, max_pos, interleaved, eps);
  p.B = B;
  p.T = T;
  p.dwq = dq_weight;
  p.dwk = dk_weight;
  p.flags = ds->flags;
  return launch_norm_rope_bwd(p, D, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

GBATTN_API int paged_qkv_append(const void* q, const void* k, const void* v,
                                const int64_t* q_strides, const int64_t* k_strides,
                                const int64_t* v_strides, const void* q_weight,
                                const void* k_weight, const float* cos_sin,
                                const int32_t* positions, void* k_pool, void* v_pool,
                                const int32_t* block_table, const int32_t* seq_lens,
                                int32_t* new_seq_lens, int block_size, int num_seqs, int Tn,
                                int Hq, int Hkv, int D, int max_blocks_per_seq,
                                int num_pool_blocks, int rot_dim, int max_pos, int interleaved,
                                float eps, void* q_out, void* stream) {
  return append(false, q, k, v, q_strides, k_strides, v_strides, q_weight, k_weight, cos_sin,
                positions, k_pool, v_pool, block_table, seq_lens, new_seq_lens, block_size,
                num_seqs, Tn, Hq, Hkv, D, max_blocks_per_seq, num_pool_blocks, rot_dim, max_pos,
                interleaved, eps, q_out, stream);
}

GBATTN_API int paged_kv4_append(const void* q, const void* k, const void* v,
                                const int64_t* q_strides, const int64_t* k_strides,
                                const int64_t* v_strides, const void* q_weight,
                                const void* k_weight, const float* cos_sin,
                                const int32_t* positions, void* kv_pool,
                                const int32_t* block_table, const int32_t* seq_lens,
                                int32_t* new_seq_lens, int block_size, int num_seqs, int Tn,
                                int Hq, int Hkv, int D, int max_blocks_per_seq,
                                int num_pool_blocks, int rot_dim, int max_pos, int interleaved,
                                float eps, void* q_out, void* stream) {
  return append(true, q, k, v, q_strides, k_strides, v_strides, q_weight, k_weight, cos_sin,
                positions, kv_pool, nullptr, block_table, seq_lens, new_seq_lens, block_size,
                num_seqs, Tn, Hq, Hkv, D, max_blocks_per_seq, num_pool_blocks, rot_dim, max_pos,
                interleaved, eps, q_out, stream);
}

GBATTN_API int paged_kv4_gather(const void* kv_pool, const int32_t* block_table,
                                const int32_t* seq_lens, int block_size, int num_seqs, int Hkv,
                                int D, int max_blocks_per_seq, int num_pool_blocks,
                                int max_seq_len, void* k_out, void* v_out, void* stream) {
  if (num_seqs < 0 || Hkv <= 0 || max_blocks_per_seq <= 0 || num_pool_blocks <= 0 ||
      max_seq_len < 0)
    return ATTN_ERR_INVALID_ARG;
  if (block_size != 16 || (D != 64 && D != 128)) return ATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_seq_len == 0) return ATTN_OK;
  if (!kv_pool || !block_table || !seq_lens || !k_out || !v_out) return ATTN_ERR_INVALID_ARG;
  if (!aligned(kv_pool, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) ||
      !aligned(block_table, 4) || !aligned(seq_lens, 4))
    return ATTN_ERR_INVALID_ARG;
  const uint64_t blocks = (static_cast<uint64_t>(max_seq_len) + 15) / 16;
  if (static_cast<unsigned __int128>(num_seqs) * Hkv * blocks >= kMaxDim ||
      static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size >= kMaxDim ||
      static_cast<uint64_t>(max_blocks_per_seq) * block_size >= kMaxDim)
    return ATTN_ERR_UNSUPPORTED;
  DeviceState* ds = nullptr;
  const int st = device_state(&ds);
  if (st != ATTN_OK) return st;
  Gather4Params p{};
  p.pool = static_cast<const uint8_t*>(kv_pool);
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.k_out = static_cast<uint16_t*>(k_out);
  p.v_out = static_cast<uint16_t*>(v_out);
  p.S = num_seqs;
  p.Hkv = Hkv;
  p.max_blocks = max_blocks_per_seq;
  p.num_pool_blocks = num_pool_blocks;
  p.max_seq_len = max_seq_len;
  p.flags = ds->flags;
  return launch_kv4_gather(p, D, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

namespace {

// Whether the row kernels' 32-bit counts of steps and rows hold a call of these sizes.
bool rows_fit(int S, int Hq, int Hkv, int Tq, int max_seq_len) {
  if (static_cast<unsigned __int128>(S) * Hq * Tq >= kMaxDim / 2) return false;
  const int64_t steps = kv4_max_steps(S, Hkv * kv4_rows(Hq, Hkv, Tq).chunks, max_seq_len);
  return static_cast<uint64_t>(steps) < kMaxDim;
}

// Attention of Tq query tokens a request by the row kernels of kv4_decode.cu.
int attend_rows(const void* q, const void* kv_pool, const int32_t* block_table,
                const int32_t* seq_lens, int S, int Hq, int Hkv, int Tq, int D, int max_blocks,
                int num_pool_blocks, int max_seq_len, int causal, float scale, void* o, float* lse,
                void* workspace, size_t workspace_bytes, void* stream) {
  const Kv4DecodeWorkspace wl = kv4_decode_workspace(S, Hq, Hkv, Tq, D, max_seq_len);
  if (wl.bytes > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < wl.bytes))
    return ATTN_ERR_INVALID_ARG;
  const Kv4Rows rows = kv4_rows(Hq, Hkv, Tq);
  DeviceState* ds = nullptr;
  const int st = device_state(&ds);
  if (st != ATTN_OK) return st;
  Kv4DecodeParams p{};
  p.q = q;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.o = o;
  p.lse = lse;
  char* ws = static_cast<char*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_lse = reinterpret_cast<float*>(ws + wl.off_part_lse);
  p.seg_first = reinterpret_cast<int*>(ws + wl.off_seg_first);
  p.seg_last = reinterpret_cast<int*>(ws + wl.off_seg_last);
  p.S = S;
  p.Hkv = Hkv;
  p.D = D;
  p.Tq = Tq;
  p.causal = causal;
  p.rows = rows.rows;
  p.piece_rows = rows.piece_rows;
  p.chunks = rows.chunks;
  p.segs = Hkv * rows.chunks;
  p.max_blocks = max_blocks;
  p.num_pool_blocks = num_pool_blocks;
  p.max_seq_len = max_seq_len;
  p.max_pieces = static_cast<int>(wl.pieces);
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.flags = ds->flags;
  p.wait_limit_ns = g_wait_limit_ns.load(std::memory_order_relaxed);
  p.withhold_copy = g_withhold_copy.load(std::memory_order_relaxed);
  return launch_kv4_decode(static_cast<const uint8_t*>(kv_pool), p, ds->num_sms,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

// Whether a chunk of Tq tokens goes to the row kernels instead of the tile kernel.  The row
// kernels' time grows with Tq and is spread over the SMs along the cache; the tile kernel
// takes the same time for 1 and for 256 tokens (one unit a query head), on as many SMs as
// there are query heads in the batch.  Measured on GB300 (us, rows / tiles):
//   16 x 32/8 heads, 6000 keys, D 128:  Tq 1: 30 / 312   16: 141 / 312   32: 266 / 312   48: 392 / 313
//   64 x 12/2 heads, 4000 keys, D 128:  Tq 1: 24 / 320   16: 146 / 321   32: 277 / 321   48: 409 / 324
//   64 x 32/8 heads, 1000 keys, D 128:  Tq 24: 194 / 212 32: 254 / 212
//   8 x 8/8 heads, 3000 keys, D 128:    Tq 16: 22 / 44   48: 38 / 44     64: 46 / 45
//   4 x 16/1 heads, 2000 keys, D 64:    Tq 16: 12 / 27   64: 26 / 27     96: 36 / 27
//   1 x 32/8 heads, 100000 keys, D 128: Tq 1: 32 / 1235  64: 499 / 1236  128: 974 / 1236  192: 1462 / 1403
// i.e. the crossing is near Tq = 30 with every SM busy and moves up as query heads are
// fewer than the 152 SMs.  Caches of up to 512 keys stay with the tiles, unless those need
// several rounds: one tile's chain is short then, and the rows take two launches and a
// workspace.  Rows / tiles (us, lengths from half the bound):
//   3 x 8/2 heads, D 64:    100 keys: Tq 4: 7.8 / 5.3   37: 9.2 / 5.3    300: 4: 7.3 / 7.9   37: 9.6 / 8.3
//                           500 keys: Tq 4: 7.2 / 9.2   16: 8.0 / 9.1    37: 9.5 / 8.2
//   1 x 32/8 heads, D 128:  300 keys: Tq 4: 8.6 / 7.8   16: 9.6 / 7.8    500: 4: 9.0 / 9.2   16: 10.4 / 9.6
//   12 x 12/2 heads, D 128: 300 keys: Tq 4: 10.0 / 10.4 16: 12.8 / 10.6  500: 4: 11.1 / 12.0 16: 13.0 / 12.1
// A few tokens on the longest of them are the exception, by up to a fifth, and single tokens
// (2.6 to 5.4 us in the one launch of a decode against 5.3 to 12), which paged_kv4_attn_decode
// is for.
// Sizes that the row kernels cannot count are the tile kernel's.
bool by_rows(int B, int Hq, int Hkv, int Tq, int max_kv_len) {
  const int64_t units = static_cast<int64_t>(B) * Hq;
  if (!rows_fit(B, Hq, Hkv, Tq, max_kv_len)) return false;
  if (max_kv_len <= 512 && units <= 152) return false;
  return Tq <= 256 && Tq * (units < 152 ? units : 152) <= 4500;
}

}  // namespace

GBATTN_API size_t paged_kv4_attn_decode_workspace_size(int num_seqs, int Hq, int Hkv, int D,
                                                       int max_seq_len) {
  if (num_seqs < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || D <= 0 || max_seq_len < 0) return 0;
  return kv4_decode_workspace(num_seqs, Hq, Hkv, 1, D, max_seq_len).bytes;
}

GBATTN_API size_t paged_kv4_attn_prefill_workspace_size(int B, int Hq, int Hkv, int Tq, int D,
                                                        int max_kv_len) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Tq <= 0 || D <= 0 || max_kv_len < 0)
    return 0;
  return by_rows(B, Hq, Hkv, Tq, max_kv_len)
             ? kv4_decode_workspace(B, Hq, Hkv, Tq, D, max_kv_len).bytes
             : 0;
}

GBATTN_API int paged_kv4_attn_decode(const void* q, const void* kv_pool,
                                     const int32_t* block_table, const int32_t* seq_lens,
                                     int block_size, int num_seqs, int Hq, int Hkv, int D,
                                     int max_blocks_per_seq, int num_pool_blocks,
                                     int max_seq_len, float scale, void* o, float* lse,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (num_seqs < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq <= 0 ||
      num_pool_blocks <= 0 || max_seq_len < 0)
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (block_size != 16 || (D != 64 && D != 128) || Hq / Hkv > 16) return ATTN_ERR_UNSUPPORTED;
  if (num_seqs == 0) return ATTN_OK;
  if (!q || !kv_pool || !block_table || !seq_lens || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(o, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(lse, 4))
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size >= kMaxDim ||
      static_cast<uint64_t>(max_blocks_per_seq) * block_size >= kMaxDim ||
      !rows_fit(num_seqs, Hq, Hkv, 1, max_seq_len))
    return ATTN_ERR_UNSUPPORTED;
  return attend_rows(q, kv_pool, block_table, seq_lens, num_seqs, Hq, Hkv, 1, D,
                     max_blocks_per_seq, num_pool_blocks, max_seq_len, 0, scale, o, lse, workspace,
                     workspace_bytes, stream);
}

GBATTN_API int paged_kv4_attn_prefill(const void* q, const void* kv_pool,
                                      const int32_t* block_table, const int32_t* kv_lens,
                                      int block_size, int B, int Hq, int Hkv, int Tq, int D,
                                      int max_blocks_per_seq, int num_pool_blocks, int max_kv_len,
                                      int causal, float scale, void* o, float* lse,
                                      void* workspace, size_t workspace_bytes, void* stream) {
  if (B < 0 || Tq < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || max_blocks_per_seq <= 0 ||
      num_pool_blocks <= 0 || max_kv_len < 0)
    return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if (block_size != 16 || (D != 64 && D != 128)) return ATTN_ERR_UNSUPPORTED;
  if (B == 0 || Tq == 0) return ATTN_OK;
  if (!q || !kv_pool || !block_table || !kv_lens || !o) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(kv_pool, 16) || !aligned(o, 16) || !aligned(block_table, 4) ||
      !aligned(kv_lens, 4) || !aligned(lse, 4))
    return ATTN_ERR_INVALID_ARG;
  const uint64_t bhq = static_cast<uint64_t>(B) * Hq;
  const uint64_t n_qpairs = (static_cast<uint64_t>(Tq) + 255) / 256;
  if (bhq >= kMaxDim || bhq * n_qpairs >= kMaxDim || bhq * Tq >= (1ull << 40) ||
      static_cast<uint64_t>(num_pool_blocks) * Hkv * block_size >= kMaxDim ||
      static_cast<uint64_t>(max_blocks_per_seq) * block_size >= kMaxDim)
    return ATTN_ERR_UNSUPPORTED;
  if (by_rows(B, Hq, Hkv, Tq, max_kv_len))
    return attend_rows(q, kv_pool, block_table, kv_lens, B, Hq, Hkv, Tq, D, max_blocks_per_seq,
                       num_pool_blocks, max_kv_len, causal, scale, o, lse, workspace,
                       workspace_bytes, stream);
  DeviceState* ds = nullptr;
  int st = device_state(&ds);
  if (st != ATTN_OK) return st;
  PFN_cuTensorMapEncodeTiled_v12000 enc = nullptr;
  if ((st = encoder(&enc)) != ATTN_OK) return st;
  CUtensorMap tmQ;
  const uint64_t row_bytes = static_cast<uint64_t>(D) * 2;
  const uint64_t strides[2] = {row_bytes, row_bytes * Tq};
  const uint32_t box[3] = {64, 128, 1};
  const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(Tq), bhq};
  if ((st = encode_bf16(enc, &tmQ, q, 3, dims, strides, box)) != ATTN_OK) return st;
  FwdParams p = fwd_params(o, lse, B, Hq, Hkv, Tq, max_kv_len, D, causal, scale, ds->flags);
  p.block_table = block_table;
  p.kv_lens = kv_lens;
  p.max_blocks = max_blocks_per_seq;
  p.num_pool_blocks = num_pool_blocks;
  p.max_kv_len = max_kv_len;
  p.kv4_pool = static_cast<const uint8_t*>(kv_pool);
  return launch_attn_fwd(tmQ, tmQ, tmQ, p, ds->num_sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}
