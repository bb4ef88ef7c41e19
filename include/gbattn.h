/*
 * gbattn.h -- C ABI of the GB300 (sm_103a) fused attention library.
 *
 * Two operations, both from the-ai.news, "Kernels de atencao rapida e fusao de
 * operadores", section "Atencao do tipo FlashAttention e atencao paginada":
 *
 *   attn_fwd           softmax attention computed block by block (scores for a
 *                      block, softmax statistics updated, output accumulated on
 *                      chip) so the T x T score matrix is never stored; i.e. the
 *                      result of the naive matmul / scale / causal mask / softmax /
 *                      matmul sequence (aiexpert.news, "Hugging Face Reduz
 *                      Sobrecarga de Atencao na Inferencia em 20-40% com Nucleos
 *                      Fundidos", second paragraph) in one kernel.
 *   paged_attn_decode  one new query token per request against a KV cache kept in
 *                      fixed-size blocks, every logical position translated
 *                      through a block table (block_size = 16, the value of the
 *                      page's vLLM example).
 *
 * Conventions for every entry point:
 *   - Tensor arguments are DEVICE pointers owned by the caller (any CUDA
 *     allocator).  The library never allocates, frees or keeps them, never
 *     synchronises the host, and enqueues work only on `stream` (a cudaStream_t
 *     passed as void*; NULL = the legacy default stream).
 *   - Tensors are contiguous, row-major, in the layouts stated below.  bf16 data
 *     pointers must be 16-byte aligned, fp32/int32 pointers 4-byte aligned.
 *   - Arguments are validated before anything is launched.  A non-OK status
 *     means nothing was enqueued (except ATTN_ERR_CUDA, see below).  There is no
 *     fallback path: unsupported inputs are an error, never a slower kernel.
 *   - Numerics: bf16 inputs, fp32 accumulation and fp32 softmax statistics; the
 *     probabilities are rounded to bf16 before they multiply V; O is rounded to
 *     bf16 (round-to-nearest-even).  LSE is the natural log of the sum of
 *     exp(scale * q.k) over the visible keys.
 *   - Thread-safe.  The first call on a device performs one-time set-up
 *     (kernel attributes, device checks).
 */
#ifndef GBATTN_H
#define GBATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ATTN_OK = 0,
    ATTN_ERR_INVALID_ARG = 1, /* null/misaligned pointer, bad size, Hq % Hkv != 0, bad scale, small workspace */
    ATTN_ERR_UNSUPPORTED = 2, /* head dim not 64/128, block_size != 16, group > 16, not an sm_103 device, size limits */
    ATTN_ERR_CUDA = 3,        /* a CUDA runtime/driver call or a launch failed; work may be partially enqueued */
    ATTN_ERR_DEVICE = 4       /* reported only by attn_device_status(): a kernel flagged bad data or a timeout */
} attn_status_t;

/* Human-readable name of a status code (static string, never NULL). */
const char *attn_status_string(int status);

/*
 * attn_fwd -- fused attention forward (prefill / full attention).
 *
 *   q   [B, Hq,  T, D] bf16      k, v [B, Hkv, T, D] bf16
 *   o   [B, Hq,  T, D] bf16 (written)
 *   lse [B, Hq,  T]    fp32 (written; may be NULL to skip)
 *
 * Query head h reads KV head h / (Hq / Hkv) (grouped-query attention; Hkv = Hq
 * is multi-head attention).  With causal != 0 query i sees keys 0..i;
 * otherwise all T keys.  scale multiplies q.k (typically 1/sqrt(D)); it must be
 * finite and > 0.  D must be 64 or 128.  B = 0 or T = 0 is a no-op.
 * Returns ATTN_OK once the kernel is enqueued.
 */
int attn_fwd(const void *q, const void *k, const void *v, void *o, float *lse, int B, int Hq,
             int Hkv, int T, int D, int causal, float scale, void *stream);

/*
 * paged_attn_prefill -- attention of a chunk of new tokens against a paged KV
 * cache (chunked prefill).  The blockwise computation of attn_fwd, with every key
 * and value position translated through the block table (same the-ai.news
 * section; block_size = 16 as in its vLLM example).
 *
 *   q             [B, Hq, Tq, D] bf16: the Tq newest tokens of each batch item
 *   k_pool/v_pool [num_pool_blocks, Hkv, block_size, D] bf16
 *   block_table   [B, max_blocks_per_seq] int32: logical block t / block_size of
 *                 item b lives in physical block block_table[b][t / block_size];
 *                 entries past ceil(kv_lens[b] / block_size) are never read
 *   kv_lens       [B] int32 (device memory): tokens in each item's cache, the Tq
 *                 new tokens' own keys and values included
 *   o             [B, Hq, Tq, D] bf16 (written)
 *   lse           [B, Hq, Tq] fp32 (written; may be NULL)
 *
 * Query i of item b is the token at logical position kv_lens[b] - Tq + i.  With
 * causal != 0 it sees keys 0 .. kv_lens[b] - Tq + i (the mask is aligned with the
 * last key); otherwise all kv_lens[b] keys.  A query that sees no key (causal
 * with kv_lens[b] < Tq) gets O = 0 and LSE = -inf.  max_kv_len bounds every
 * kv_lens[b].  block_size must be 16 and D 64 or 128.  Per-item data is checked
 * on the device: a kv_lens[b] outside [0, min(max_kv_len, max_blocks_per_seq *
 * block_size)] makes that item's O and LSE NaN and sets flag bit 2; a block id
 * outside [0, num_pool_blocks) is read as block 0 and sets flag bit 4 (that
 * item's output is then unspecified).  Pool slots past kv_lens[b] may hold any
 * bits, NaN included: they never reach the output.
 */
int paged_attn_prefill(const void *q, const void *k_pool, const void *v_pool,
                       const int32_t *block_table, const int32_t *kv_lens, int block_size, int B,
                       int Hq, int Hkv, int Tq, int D, int max_blocks_per_seq,
                       int num_pool_blocks, int max_kv_len, int causal, float scale, void *o,
                       float *lse, void *stream);

/*
 * Bytes of scratch workspace paged_attn_decode needs for these sizes.  The
 * decode cuts the batch's (request, KV head, 16-token block) sequence into equal
 * ranges of at least 256 tokens; each range that meets a request's cache yields
 * one partial output (D fp32) and LSE per query head, at most
 * ceil(max_seq_len / 256) + 1 per (request, query head).  Depends only on the
 * arguments; the block size is not one of them (it is fixed at 16 and checked by
 * paged_attn_decode).
 */
size_t paged_attn_decode_workspace_size(int num_seqs, int Hq, int D, int max_seq_len);

/*
 * paged_attn_decode -- one query token per request against a paged KV cache.
 *
 *   q            [num_seqs, Hq, D] bf16  (the newest token of each request)
 *   k_pool/v_pool [num_pool_blocks, Hkv, block_size, D] bf16
 *   block_table  [num_seqs, max_blocks_per_seq] int32: logical block b of
 *                request r lives in physical block block_table[r][b]; entries
 *                past ceil(seq_lens[r] / block_size) are never read
 *   seq_lens     [num_seqs] int32 (device memory): tokens in each request's
 *                cache, the new token's own K/V included
 *   o            [num_seqs, Hq, D] bf16 (written)
 *   lse          [num_seqs, Hq] fp32 (written; may be NULL)
 *   workspace    >= paged_attn_decode_workspace_size(...) bytes of device
 *                memory, 256-byte aligned; its contents need no initialisation
 *                and are scratch after the call
 *
 * The query of request r attends to all seq_lens[r] cached tokens.  A request
 * with seq_lens[r] == 0 gets O = 0 and LSE = -inf.  max_seq_len bounds every
 * seq_lens[r] (it sizes the workspace).  The split of the work depends on the
 * lengths of the whole batch, never on where the blocks sit in the pool: the
 * same inputs give the same bits, whatever the placement.  block_size must be 16, D 64 or 128,
 * Hq / Hkv <= 16.  Per-request data is checked on the device: a length outside
 * [0, min(max_seq_len, max_blocks_per_seq * block_size)] or a block id outside
 * [0, num_pool_blocks) makes that request's O and LSE NaN and sets a flag that
 * attn_device_status() reports; the kernel never traps.
 */
int paged_attn_decode(const void *q, const void *k_pool, const void *v_pool,
                      const int32_t *block_table, const int32_t *seq_lens, int block_size,
                      int num_seqs, int Hq, int Hkv, int D, int max_blocks_per_seq,
                      int num_pool_blocks, int max_seq_len, float scale, void *o, float *lse,
                      void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of device scratch paged_attn_decode_noalloc reserves on each device. */
#define GBATTN_DECODE_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)

/*
 * paged_attn_decode_noalloc -- paged_attn_decode without a caller workspace.
 *
 * The pages have no counterpart of this entry point; it exists for callers that
 * cannot allocate device memory at the point where they decode: code running
 * inside an allocator's own hooks, a host application that owns every device
 * allocation and hands out none, or a latency-critical loop that must never
 * enter the allocator.  Such a caller still owns and passes every input and
 * output (same arguments, layouts and checks as paged_attn_decode); only the
 * split-KV scratch comes from the library, from one fixed array of
 * GBATTN_DECODE_NOALLOC_SCRATCH_BYTES (16 MiB) in the library's device image.
 * Every GPU on which the library's kernels are loaded holds that array until
 * the process exits.  The call itself allocates nothing: no cudaMalloc, no
 * cudaFree, no allocating library routine.
 *
 *   - Sizes whose scratch, paged_attn_decode_workspace_size(num_seqs, Hq, D,
 *     max_seq_len), exceeds the array return ATTN_ERR_UNSUPPORTED before any
 *     work is enqueued (at D = 128 that is about 32,000 (request, query head,
 *     range) partial results; 64 requests x 12 heads x 8192 tokens need
 *     13.1 MB).
 *   - The first call on a device looks up the array's device address (once,
 *     with that device current); make that first call before any stream
 *     capture begins.
 *   - All calls on a device share the one array and it keeps whatever the last
 *     call wrote.  Nothing in it needs to start at zero: each call writes every
 *     scratch element it later reads.  Calls whose executions overlap on the GPU
 *     (different streams with no ordering between them) race on the array and
 *     give wrong results: order them on one stream or with events.
 */
int paged_attn_decode_noalloc(const void *q, const void *k_pool, const void *v_pool,
                              const int32_t *block_table, const int32_t *seq_lens, int block_size,
                              int num_seqs, int Hq, int Hkv, int D, int max_blocks_per_seq,
                              int num_pool_blocks, int max_seq_len, float scale, void *o,
                              float *lse, void *stream);

/*
 * Synchronises the current device (every stream), then reads and clears the
 * library's device flag word.  The word is one per device, shared by every
 * stream and every caller of the library in the process: a flag raised by any
 * kernel of this library on that device stays set until the next call of this
 * function, which reports and clears it for everyone.  *flags (if not NULL) receives the raw bits: 1 = a bounded wait in
 * a kernel timed out, 2 = a decode request had an invalid length, 4 = a decode
 * block id was out of range, 8 = a position lay outside the rotation table, 16 = a tree or
 * a path was invalid, 32 = a token was to be drawn from a distribution without mass.
 * Returns ATTN_ERR_DEVICE if any bit was set,
 * ATTN_ERR_CUDA if the synchronisation failed, else ATTN_OK.
 */
int attn_device_status(unsigned int *flags);

/*
 * paged_kv_append -- writes Tn new tokens per request into the paged KV cache (the
 * cache "grows one token at a time", same the-ai.news section).
 *
 *   k_new, v_new  [num_seqs, Hkv, Tn, D] bf16: the new tokens' keys and values
 *   k_pool/v_pool [num_pool_blocks, Hkv, block_size, D] bf16 (written in place)
 *   block_table   [num_seqs, max_blocks_per_seq] int32; the blocks that the new
 *                 positions fall into must already be assigned
 *   seq_lens      [num_seqs] int32 (device): tokens already cached, L_r
 *   new_seq_lens  [num_seqs] int32 (device, may be NULL): receives L_r + Tn; it
 *                 must not overlap seq_lens
 *
 * Token t of request r goes to logical position L_r + t, i.e. physical block
 * block_table[r][(L_r + t) / 16], slot (L_r + t) % 16.  The copy is exact (bits
 * in = bits out).  Device-side checks: L_r < 0 or L_r + Tn > max_blocks_per_seq *
 * block_size skips the request, sets flag bit 2 and writes L_r unchanged to
 * new_seq_lens; a block id outside the pool skips that token and sets flag bit 4.
 * block_size must be 16, D 64 or 128.
 */
int paged_kv_append(const void *k_new, const void *v_new, void *k_pool, void *v_pool,
                    const int32_t *block_table, const int32_t *seq_lens, int32_t *new_seq_lens,
                    int block_size, int num_seqs, int Hkv, int Tn, int D, int max_blocks_per_seq,
                    int num_pool_blocks, void *stream);

/*
 * paged_kv_gather -- copies each request's cached keys (or values) out of the
 * paged pool in logical order, with the same block-table translation and the
 * same TMA box copies that the attention kernels use.
 *
 *   pool          [num_pool_blocks, Hkv, block_size, D] bf16
 *   block_table   [num_seqs, max_blocks_per_seq] int32
 *   seq_lens      [num_seqs] int32 (device)
 *   out           [num_seqs, Hkv, max_seq_len, D] bf16: out[r][h][t] = the row of
 *                 token t < seq_lens[r]; rows t >= seq_lens[r] are not written
 *
 * Device-side checks: a length outside [0, min(max_seq_len, max_blocks_per_seq
 * * block_size)] skips the request and sets flag bit 2; a block id outside the
 * pool writes NaN rows for that block and sets flag bit 4.
 */
int paged_kv_gather(const void *pool, const int32_t *block_table, const int32_t *seq_lens,
                    int block_size, int num_seqs, int Hkv, int D, int max_blocks_per_seq,
                    int num_pool_blocks, int max_seq_len, void *out, void *stream);

/*
 * qkv_norm_rope -- from the rows of a QKV projection to the operands of attn_fwd:
 * RMS norm of every query and key head, rotation by position, and the move to
 * [B, H, T, D], in one pass.
 *
 *   q [B, T, Hq, D], k, v [B, T, Hkv, D] bf16, strided: *_strides points at three
 *                 HOST values, the batch, token and head strides in elements
 *                 (the channels are contiguous).  Views of one fused projection
 *                 buffer are the usual case; a stride of 0 repeats an input.
 *   q_weight, k_weight [D] bf16, or NULL: that operand is not normalised
 *   cos_sin       [max_pos, rot_dim] fp32, or NULL with rot_dim = 0: no rotation.
 *                 Row p holds the rot_dim / 2 cosines, then the sines, of position
 *                 p (any factor that scales them is applied with them)
 *   positions     [B, T] int32, or NULL: token t sits at position t
 *   q_out [B, Hq, T, D], k_out, v_out [B, Hkv, T, D] bf16 (written)
 *
 * Per row x of D channels: x * rsqrt(mean(x^2) + eps) * weight, then the first
 * rot_dim channels turn as rot_dim / 2 planes, (i, i + rot_dim / 2) or, with
 * interleaved = 1, (2 i, 2 i + 1): a, b -> a cos - b sin, b cos + a sin.  fp32
 * throughout, rounded to bf16 once.  v is copied.  Any of q, k and v may be NULL
 * together with its output; that operand is left out.  Outputs must not overlap
 * inputs.  D must be 64 or 128, rot_dim a multiple of 8 in [0, D], eps finite and
 * > 0, strides non-negative multiples of 8.  B = 0 or T = 0 is a no-op.
 * A position outside [0, max_pos) makes that token's q_out and k_out rows NaN and
 * sets flag bit 8.
 */
int qkv_norm_rope(const void *q, const void *k, const void *v, const int64_t *q_strides,
                  const int64_t *k_strides, const int64_t *v_strides, const void *q_weight,
                  const void *k_weight, const float *cos_sin, const int32_t *positions, int B,
                  int T, int Hq, int Hkv, int D, int rot_dim, int max_pos, int interleaved,
                  float eps, void *q_out, void *k_out, void *v_out, void *stream);

/* Bytes of scratch qkv_norm_rope_bwd needs for these sizes (0 when B or T is 0). */
size_t qkv_norm_rope_bwd_workspace_size(int B, int T, int D);

/*
 * qkv_norm_rope_bwd -- gradients of qkv_norm_rope.
 *
 *   dq_out [B, Hq, T, D], dk_out, dv_out [B, Hkv, T, D] bf16: gradients of the
 *                 outputs; NULL leaves that operand out
 *   q, k          the forward's inputs with their strides; read only where there is
 *                 a weight, and may be NULL otherwise
 *   dq, dk, dv    gradients of the inputs (written), [B, T, H, D] bf16 with strides
 *                 as above; the layout must give every element a place of its own
 *   dq_weight, dk_weight [D] fp32 (written), required with the weight and NULL
 *                 without it: summed over tokens and heads in an order that depends
 *                 on the sizes and on which operands take part, so they are the
 *                 same bits on every run.  They
 *                 are written (as zeros) for B = 0 or T = 0 too
 *   workspace     >= qkv_norm_rope_bwd_workspace_size(...) bytes of device memory,
 *                 16-byte aligned, needed when there is a weight; no initialisation
 *
 * Everything else as in qkv_norm_rope.  A position outside the table makes that
 * token's dq and dk rows and the weight gradients NaN and sets flag bit 8.
 */
int qkv_norm_rope_bwd(const void *dq_out, const void *dk_out, const void *dv_out, const void *q,
                      const void *k, const int64_t *q_strides, const int64_t *k_strides,
                      const void *q_weight, const void *k_weight, const float *cos_sin,
                      const int32_t *positions, int B, int T, int Hq, int Hkv, int D, int rot_dim,
                      int max_pos, int interleaved, float eps, void *dq, void *dk, void *dv,
                      const int64_t *dq_strides, const int64_t *dk_strides,
                      const int64_t *dv_strides, float *dq_weight, float *dk_weight,
                      void *workspace, size_t workspace_bytes, void *stream);

/*
 * paged_qkv_append -- paged_kv_append with qkv_norm_rope on the way: the Tn new
 * tokens of each request are normalised and rotated, K and V go into the paged
 * cache, and the queries come out as the attention entry points read them.
 *
 *   q [num_seqs, Tn, Hq, D] (NULL together with q_out: no queries), k, v
 *                 [num_seqs, Tn, Hkv, D] bf16, strided as in qkv_norm_rope
 *   positions     [num_seqs, Tn] int32, or NULL: token t of request r is rotated by
 *                 its place in the cache, seq_lens[r] + t
 *   q_out         [num_seqs, Hq, Tn, D] bf16 (written); for Tn = 1 that is
 *                 paged_attn_decode's q
 *   k_pool/v_pool, block_table, seq_lens, new_seq_lens, block_size as in
 *                 paged_kv_append (Tn = 0 copies the lengths to new_seq_lens and does
 *                 nothing else); the rest as in qkv_norm_rope
 *
 * Device-side checks: a length with no room for Tn more tokens skips the request
 * (its q_out rows become NaN, new_seq_lens keeps the length) and sets flag bit 2; a
 * block id outside the pool skips that token's K and V and sets flag bit 4; a
 * position outside the table skips that token's K and V, makes its q_out rows NaN
 * and sets flag bit 8.  The slots written in one call must be distinct: two requests
 * may share blocks only where neither appends.
 */
int paged_qkv_append(const void *q, const void *k, const void *v, const int64_t *q_strides,
                     const int64_t *k_strides, const int64_t *v_strides, const void *q_weight,
                     const void *k_weight, const float *cos_sin, const int32_t *positions,
                     void *k_pool, void *v_pool, const int32_t *block_table,
                     const int32_t *seq_lens, int32_t *new_seq_lens, int block_size, int num_seqs,
                     int Tn, int Hq, int Hkv, int D, int max_blocks_per_seq, int num_pool_blocks,
                     int rot_dim, int max_pos, int interleaved, float eps, void *q_out,
                     void *stream);

/*
 * The 4-bit paged KV cache.  A pool is [num_pool_blocks, Hkv, 18 D] bytes, 16-byte
 * aligned; one chunk of 18 D bytes holds a block's 16 tokens of one KV head:
 *
 *   K codes [16][D / 2], K scales [16][D / 32] bf16, V codes, V scales alike
 *
 * 32 consecutive channels share a scale s: the largest magnitude / 7 rounded to 5
 * significant bits.  A channel x is held as n + 8 with n = x / s rounded to even and
 * kept in [-7, 7], and stands for n * s, which is a bf16 exactly (code 0 reads as
 * -8).  A NaN or infinity makes its group read as NaN.  Two codes share a byte, the
 * even position in the low half; channel c of a K row is at position
 * (c % 32 / 8 * (D / 32) + c / 32) * 8 + c % 8, of a V row at position
 * (c % 32 / 4 * (D / 32) + c / 32) * 4 + c % 4.
 * A block takes 28 % of the memory of its bf16 form (2304 bytes at D = 128).
 */

/*
 * paged_kv4_append -- paged_qkv_append into the 4-bit cache: keys are normalised,
 * rotated and rounded to bf16, then quantised; values are quantised as they are.
 * With rot_dim = 0 and no weights it quantises keys that are ready.  kv_pool takes
 * the place of the two bf16 pools; everything else as in paged_qkv_append.
 */
int paged_kv4_append(const void *q, const void *k, const void *v, const int64_t *q_strides,
                     const int64_t *k_strides, const int64_t *v_strides, const void *q_weight,
                     const void *k_weight, const float *cos_sin, const int32_t *positions,
                     void *kv_pool, const int32_t *block_table, const int32_t *seq_lens,
                     int32_t *new_seq_lens, int block_size, int num_seqs, int Tn, int Hq, int Hkv,
                     int D, int max_blocks_per_seq, int num_pool_blocks, int rot_dim, int max_pos,
                     int interleaved, float eps, void *q_out, void *stream);

/*
 * paged_kv4_gather -- the values the 4-bit cache holds, in logical order.
 *
 *   kv_pool       [num_pool_blocks, Hkv, 18 D] bytes
 *   k_out, v_out  [num_seqs, Hkv, max_seq_len, D] bf16: row t < seq_lens[r] of
 *                 request r; rows past it are not written
 *
 * Everything else, the device-side checks included, as in paged_kv_gather.
 */
int paged_kv4_gather(const void *kv_pool, const int32_t *block_table, const int32_t *seq_lens,
                     int block_size, int num_seqs, int Hkv, int D, int max_blocks_per_seq,
                     int num_pool_blocks, int max_seq_len, void *k_out, void *v_out,
                     void *stream);

/*
 * Bytes of scratch workspace paged_kv4_attn_decode needs for these sizes: one partial
 * output (D fp32) and LSE per query head for each of at most 2048 + num_seqs * Hkv
 * pieces of the batch; 0 for short caches, which need none.
 */
size_t paged_kv4_attn_decode_workspace_size(int num_seqs, int Hq, int Hkv, int D,
                                            int max_seq_len);

/*
 * Bytes of scratch workspace paged_kv4_attn_prefill needs for these sizes: 0 for
 * chunks long enough for its tile kernel, else partial results as in the decode.
 */
size_t paged_kv4_attn_prefill_workspace_size(int B, int Hq, int Hkv, int Tq, int D,
                                             int max_kv_len);

/*
 * paged_kv4_attn_decode -- paged_attn_decode over the 4-bit cache: the attention of
 * one query token per request over the values that paged_kv4_gather returns.
 *
 *   kv_pool       [num_pool_blocks, Hkv, 18 D] bytes
 *   workspace     >= paged_kv4_attn_decode_workspace_size(...) bytes, 256-byte aligned
 *                 (may be NULL where that is 0); no initialisation
 *
 * Everything else, the device-side checks included, as in paged_attn_decode.  A NaN in
 * a key of the cache makes that request's O and LSE NaN for the heads that read it, a
 * NaN in a value the 32 channels of O that share its scale.
 */
int paged_kv4_attn_decode(const void *q, const void *kv_pool, const int32_t *block_table,
                          const int32_t *seq_lens, int block_size, int num_seqs, int Hq, int Hkv,
                          int D, int max_blocks_per_seq, int num_pool_blocks, int max_seq_len,
                          float scale, void *o, float *lse, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * paged_kv4_attn_prefill -- paged_attn_prefill over the 4-bit cache: the attention of
 * the Tq newest tokens of each item over the values that paged_kv4_gather returns.
 * The values are bf16 exactly, so the kernel computes with them as they are (long chunks
 * hold values of groups whose scale is below 2^-123 to within 2^-128).
 *
 *   kv_pool       [num_pool_blocks, Hkv, 18 D] bytes
 *   workspace     >= paged_kv4_attn_prefill_workspace_size(...) bytes, 256-byte
 *                 aligned (may be NULL where that is 0); no initialisation
 *
 * Short chunks (a few drafted tokens) run as a decode of group * Tq query rows a KV
 * head, split along the cache; longer ones as 128-row tiles.  An invalid block id makes
 * that item's O unspecified (NaN in short chunks) and sets flag bit 4.
 * Everything else, the device-side checks included, as in paged_attn_prefill.  Slots
 * past kv_lens[b] may hold any bits.  A NaN in a key of the cache makes O and LSE NaN
 * for the queries that see it; a NaN in a value may reach O of every query of its item
 * and KV head, of those too that causal hides it from.
 */
int paged_kv4_attn_prefill(const void *q, const void *kv_pool, const int32_t *block_table,
                           const int32_t *kv_lens, int block_size, int B, int Hq, int Hkv, int Tq,
                           int D, int max_blocks_per_seq, int num_pool_blocks, int max_kv_len,
                           int causal, float scale, void *o, float *lse, void *workspace,
                           size_t workspace_bytes, void *stream);

/*
 * Trees of drafted tokens.  A step of decoding with drafted tokens appends the nodes of a
 * tree behind each request's cache (paged_qkv_append or paged_kv_append; a node's position
 * for its rotation is the request's length + the node's depth), attends to them with
 * paged_attn_tree, decides with draft_verify which of them the target model accepts, and
 * moves the accepted nodes' rows together with paged_kv_keep.
 *
 * A tree has at most GBATTN_TREE_MAX_NODES nodes.  parents [num_seqs, Tn] int32 gives the
 * parent of each node, -1 for a root; a parent comes before its children (parents[r][i] <
 * i).  A chain of drafts is the tree with parents[r][i] = i - 1.  tree_lens [num_seqs]
 * int32 (NULL: Tn for every request) says how many of the Tn places hold nodes.
 */
#define GBATTN_TREE_MAX_NODES 256

/*
 * Bytes of scratch workspace paged_attn_tree needs for these sizes (0 for sizes that need
 * none): partial outputs (D fp32) and LSEs of the query rows that share a cache cut between
 * two CTAs.
 */
size_t paged_attn_tree_workspace_size(int num_seqs, int Tn, int Hq, int Hkv, int D,
                                      int max_seq_len);

/*
 * paged_attn_tree -- attention of the nodes of a tree of drafted tokens per request against
 * the paged cache: paged_attn_prefill with the tree in the place of the causal chunk.
 *
 *   q             [num_seqs, Hq, Tn, D] bf16: the nodes' queries
 *   k_pool/v_pool [num_pool_blocks, Hkv, block_size, D] bf16
 *   block_table   [num_seqs, max_blocks_per_seq] int32
 *   seq_lens      [num_seqs] int32 (device): tokens cached before the tree, L_r; node i's
 *                 key and value are at logical position L_r + i
 *   parents       [num_seqs, Tn] int32, tree_lens [num_seqs] int32 or NULL: see above
 *   o             [num_seqs, Hq, Tn, D] bf16 (written)
 *   lse           [num_seqs, Hq, Tn] fp32 (written; may be NULL)
 *   workspace     >= paged_attn_tree_workspace_size(...) bytes, 256-byte aligned (may be
 *                 NULL where that is 0); no initialisation
 *
 * Node i sees the L_r cached tokens, its ancestors and itself.  Places past a tree's nodes
 * get O = 0 and LSE = -inf; what is cached for them is not read.  max_seq_len bounds every
 * L_r + tree_lens[r].  Tn is at most GBATTN_TREE_MAX_NODES, block_size 16, D 64 or 128, Hq /
 * Hkv <= 128; with s = the segments num_seqs * Hkv (times 2, 3, .. where the nodes' rows make
 * more than 16, 32, .. tiles of 128), s * (max_seq_len / 128 + 3) * 20 has to stay below 2^31
 * (ATTN_ERR_UNSUPPORTED otherwise).  The split of the work depends on the lengths
 * of the whole batch, never on the blocks' places: the same inputs give the same bits.
 *
 * Device-side checks: a length or a number of nodes outside its bounds, or L_r +
 * tree_lens[r] outside [0, min(max_seq_len, max_blocks_per_seq * block_size)], makes that
 * request's O and LSE NaN and sets flag bit 2; a parent outside [-1, i) makes those of all
 * its nodes NaN and sets flag bit 16.  A block id outside the pool is read as block 0 and sets flag bit 4 (that
 * request's output is then unspecified).  Slots past the tree may hold any bits.  A NaN or an
 * infinity in a value may reach O of every node of its request, of those too that do not see it
 * (in a key it does not).
 */
int paged_attn_tree(const void *q, const void *k_pool, const void *v_pool,
                    const int32_t *block_table, const int32_t *seq_lens, const int32_t *parents,
                    const int32_t *tree_lens, int block_size, int num_seqs, int Tn, int Hq,
                    int Hkv, int D, int max_blocks_per_seq, int num_pool_blocks, int max_seq_len,
                    float scale, void *o, float *lse, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * draft_verify -- which drafted tokens the target model accepts, and the token after them,
 * so that what is put out is distributed as the target's own draws would be.
 *
 *   target_probs  [num_seqs, Tn, V] fp32 (prob_type 0) or bf16 (1): row i is the target's
 *                 distribution of the token after node i
 *   draft_probs   the same type, or NULL: row i is the distribution that node i's children
 *                 were drawn from, independently.  NULL: they were put forward without a
 *                 draw (the likeliest few, say)
 *   *_strides     two HOST values, the strides of requests and of nodes in elements; the V
 *                 probabilities of a row are contiguous
 *   tokens        [num_seqs, Tn] int32: the nodes' tokens.  Node 0 is the token that the
 *                 tree hangs from: it stands already, and its entry is not read
 *   parents, tree_lens  as above
 *   uniforms      [num_seqs, Tn] fp32 random numbers in [0, 1): number i > 0 decides on
 *                 node i, number 0 draws the last token
 *   tokens_out    [num_seqs, Tn] int32 (written): the accepted nodes' tokens, root left out,
 *                 then the last token, then -1
 *   path          [num_seqs, Tn] int32 (written): the accepted nodes, from node 0 down, then
 *                 -1
 *   counts        [num_seqs] int32 (written): how many nodes stand, and so how many tokens
 *                 are put out
 *
 * From node 0 on, with w = p (the target's row of the node reached), W = 1: the node's
 * children are tried in the order of their numbers.  Child i with token x stands if
 * u_i q(x) W < w(x) (q: the draft's row; without one q(x) = 1 and q = 0 elsewhere), and the
 * search goes on from there.  If it falls, w becomes max(w - W q, 0) and W its sum, unless
 * that is 0, in which case both stay.  Where no child stands, the last token is the first x
 * whose w(0) + .. + w(x) is above u_0 times the sum of w (-1 and flag bit 32 if the sum is
 * 0).  Probabilities and random numbers are taken to [0, 1] (NaN as 0).  Tests take them as
 * multiples of 2^-62, sums over w as multiples of 2^-44 (each value off by less than one of
 * them), so that sums do not depend on an order; a row may sum to anything below 4.  (Sums wrap
 * from there on: the last token of such a row is any of the V, or -1 with flag bit 32.)  Tokens
 * outside [0, V) have probability 0.
 *
 * tokens_out, path and counts may be tokens, parents and tree_lens.
 *
 * A request without nodes gets count 0.  Device-side checks: a number of nodes outside
 * [0, Tn] (flag bit 2) or a parent outside [-1, i) (flag bit 16) gives count 0 as well.
 * Tn is at most GBATTN_TREE_MAX_NODES, V below 2^30; strides are non-negative.
 */
int draft_verify(const void *target_probs, const void *draft_probs, const int64_t *target_strides,
                 const int64_t *draft_strides, int prob_type, const int32_t *tokens,
                 const int32_t *parents, const float *uniforms, const int32_t *tree_lens,
                 int num_seqs, int Tn, int V, int32_t *tokens_out, int32_t *path, int32_t *counts,
                 void *stream);

/*
 * paged_kv_keep -- keeps chosen rows behind each request's cache and moves them together:
 * the row at logical position L_r + path[r][j] goes to L_r + j for every j < counts[r], key
 * and value, every KV head, in every layer.
 *
 *   k_pools, v_pools  HOST arrays of num_layers device pointers, each to a pool
 *                 [num_pool_blocks, Hkv, block_size, D] bf16 (changed in place); the pools
 *                 must not overlap (ATTN_ERR_INVALID_ARG: rows would move twice)
 *   block_table   [num_seqs, max_blocks_per_seq] int32, shared by the layers
 *   seq_lens      [num_seqs] int32 (device): L_r, the tokens before those rows
 *   path          [num_seqs, path_len] int32: strictly increasing (entries past counts[r]
 *                 are not read)
 *   counts        [num_seqs] int32, at most path_len
 *   new_seq_lens  [num_seqs] int32 (may be NULL): receives L_r + counts[r]; it must not
 *                 overlap another operand
 *
 * Rows that stay in place are not touched, nor is any other row.  path_len is at most
 * GBATTN_TREE_MAX_NODES.  Device-side checks: a length or count out of bounds, or a last row
 * past max_blocks_per_seq * block_size (flag bit 2), or a path that does not increase (flag
 * bit 16) skips the request and writes L_r unchanged to new_seq_lens; a move from or to a
 * block id outside the pool is skipped and sets flag bit 4.  Two requests may share blocks
 * only below their lengths.
 */
int paged_kv_keep(void *const *k_pools, void *const *v_pools, int num_layers,
                  const int32_t *block_table, const int32_t *seq_lens, const int32_t *path,
                  const int32_t *counts, int32_t *new_seq_lens, int block_size, int num_seqs,
                  int path_len, int Hkv, int D, int max_blocks_per_seq, int num_pool_blocks,
                  void *stream);

/*
 * Test hook for the kernels' failure detection (not for production use).
 * Kernels launched after this call use wait_limit_ns as the limit, in
 * nanoseconds, of every pipeline wait (0 restores the default of 2 s).  With
 * withhold_copy = 1 the copy warp of every CTA of the next kernels skips its
 * first data copy, so a consumer's wait for it is certain to run out: the
 * waiting role raises flag bit 1, tells the CTA's other roles to stop, lets the
 * copies and MMAs already in flight finish, and the kernel returns with
 * unspecified outputs; attn_device_status() then reports ATTN_ERR_DEVICE.  No
 * fault, trap or hang is involved.  Call attn_test_set_failure(0, 0) to restore
 * normal operation.  Process-wide; not meant for use while other threads launch
 * kernels of this library.  Returns ATTN_OK, or ATTN_ERR_INVALID_ARG if
 * withhold_copy is not 0 or 1.
 */
int attn_test_set_failure(unsigned long long wait_limit_ns, int withhold_copy);

/* Library version as MAJOR * 10000 + MINOR * 100 + PATCH. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GBATTN_H */
