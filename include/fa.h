/*
 * fa.h — C ABI of the B200 (sm_100a) exact-attention library.
 *
 * The operation is exact scaled-dot-product attention, O = softmax(Q K^T * scale) V,
 * computed tile by tile with the online-softmax recurrence (running maximum m, sum
 * l = sum_j e^{s_j - m}, numerator u = sum_j e^{s_j - m} v_j; l and u rescaled by
 * e^{m - m'} whenever a tile raises the maximum; output u / l), so the Nq x Nkv score
 * matrix never reaches device memory.
 *   - Definition: "Autoatención, kernels CUDA y FlashAttention", §1 (Scores = QK^T /
 *     sqrt(d_k); row softmax; Attention(Q,K,V) = softmax(QK^T / sqrt(d_k)) V; heads in
 *     parallel).
 *   - Blocked evaluation and recomputation in the backward pass: same page, §3
 *     ("Procesamiento por bloques", "El truco de Softmax en línea", "Recálculo durante
 *     la retropropagación").
 *   - The (m, l, u) recurrence and why block results cannot be averaged: "FlashAttention"
 *     (paweldubiel.com notes), "No basta con promediar los resultados de los bloques".
 *   - GQA: same page, "Mecanismo y detalles", last paragraph.
 *   - Paged KV cache and block table: "Kernels de atención rápida y fusión de operadores"
 *     (the-ai.news), "Atención tipo FlashAttention y atención paginada".
 *
 * Conventions common to every entry point
 *   - All tensor pointers are DEVICE pointers to contiguous row-major arrays, at least
 *     16-byte aligned.  The caller owns every buffer, workspaces included; the library
 *     never allocates device memory.  Its only state between calls is the process-wide
 *     settings of fa_set_wait_limit_ns and fa_set_decode_split and, for
 *     fa_paged_decode_noalloc, the cached address of its scratch array; and, for kernels that
 *     need launch attributes, on which devices these have been set.
 *   - Calls are asynchronous on `stream` (a cudaStream_t passed as void*; NULL is the
 *     legacy default stream).  FA_OK means the launch was accepted.  Faults that
 *     happen while the kernel runs surface at the caller's next synchronisation.
 *   - Arguments are validated on the host before anything is launched.  Nothing is
 *     launched when a call returns an error.  There is no CPU fallback and no
 *     alternative backend: unsupported input is an error (FA_ERR_UNSUPPORTED).
 *   - Layouts: q, o [B, Hq, Nq, d]; k, v [B, Hkv, Nkv, d]; lse [B, Hq, Nq] fp32.
 *     Query head h reads key/value head h / (Hq / Hkv) (GQA, contiguous groups).
 *   - lse = m + ln(l) of the scaled scores (natural log), one per query row.
 *   - Causal masking is bottom-right aligned: query i may attend keys
 *     j <= i + (Nkv - Nq).  causal with Nq > Nkv is rejected.
 *   - Every waiting loop inside the kernels is bounded; a wait that runs out sets a
 *     device status word (read with fa_device_status) and the kernel returns early.
 */
#ifndef FA_H_
#define FA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, misalignment, bad shape */
  FA_ERR_UNSUPPORTED = 2,   /* valid but not built: head dim, dtype, block size */
  FA_ERR_CUDA = 3,          /* a CUDA runtime/driver call failed at launch time */
  FA_ERR_WORKSPACE = 4,     /* workspace missing or smaller than the size query says */
  FA_ERR_DEVICE_TIMEOUT = 5 /* a bounded in-kernel wait ran out (see fa_device_status) */
} fa_status;

typedef enum { FA_DTYPE_F32 = 0, FA_DTYPE_BF16 = 1 } fa_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char* fa_status_string(fa_status s);

/* Library version as an integer (major*10000 + minor*100 + patch). */
int fa_version(void);

/*
 * fa_fwd — forward pass.  Writes O (dtype `dtype`) and lse (fp32).
 *   q [B,Hq,Nq,d], k and v [B,Hkv,Nkv,d], o [B,Hq,Nq,d]: dtype `dtype`.
 *   lse [B,Hq,Nq] fp32, may not be NULL.
 *   dtype BF16: d in {64, 96, 128, 256}, tcgen05 tensor-core kernels, fp32 accumulation,
 *   P rounded to bf16 before P·V (d == 96 runs the d == 128 kernel on zero-filled
 *   columns; d == 256 has its own one-query-tile kernel).  dtype F32: fp32 SIMT kernel,
 *   d == 64.
 *   scale > 0 (usually 1/sqrt(d)); causal 0 or 1.
 * Errors: FA_ERR_INVALID_ARG (null/misaligned pointer, size <= 0, Hq % Hkv != 0,
 * scale not finite or <= 0, causal && Nq > Nkv); FA_ERR_UNSUPPORTED (other d or dtype).
 */
fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse,
                 int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale, int causal,
                 fa_dtype dtype, void* stream);

/*
 * fa_bwd_workspace_size — bytes of device workspace fa_bwd needs: an fp32 dQ
 * accumulator [B,Hq,Nq,d], then lse in base 2 and D_i = sum_c dO_ic O_ic, each
 * [B,Hq,ceil(Nq/128)*128] fp32; every region 256-byte aligned.  Returns 0 for invalid
 * sizes.
 */
size_t fa_bwd_workspace_size(int B, int Hq, int Nq, int d);

/*
 * fa_bwd — backward pass of fa_fwd, recomputing the score tiles from lse instead of
 * storing them ("Recálculo durante la retropropagación").
 *   q, k, v, o, dO: dtype `dtype` (BF16 only), layouts as in fa_fwd; lse from fa_fwd.
 *   dq [B,Hq,Nq,d], dk and dv [B,Hkv,Nkv,d] of dtype `grad_dtype` (F32 or BF16); dk
 *   and dv are summed over the Hq/Hkv query heads that share a key/value head.
 *   workspace: at least fa_bwd_workspace_size(B,Hq,Nq,d) bytes, 256-byte aligned;
 *   its contents on entry do not matter.
 *   dtype BF16: d in {64, 96, 128, 256}, tensor-core kernels (d == 96 on the d == 128
 *   kernel; d == 256 on a kernel whose CTAs each own one half of the head dimension and
 *   recompute the full-d score tiles).  dtype F32: d == 64 and grad_dtype F32, CUDA-core
 *   kernels (fp32 products throughout).
 * Errors: as fa_fwd, plus FA_ERR_WORKSPACE.
 */
fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
                 const void* dO, void* dq, void* dk, void* dv, fa_dtype grad_dtype,
                 int B, int Hq, int Hkv, int Nq, int Nkv, int d, float scale, int causal,
                 fa_dtype dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_paged_decode_workspace_size — bytes of device workspace fa_paged_decode needs
 * for the split-KV partial results: fp32 O [R,Hq,splits,d] and lse [R,Hq,splits], each
 * 256-byte aligned, with splits = ceil(max_blocks_per_seq / split size) for the split
 * size in force (see fa_set_decode_split).  Returns 0 for invalid sizes.
 */
size_t fa_paged_decode_workspace_size(int R, int Hq, int d, int max_blocks_per_seq, int block_size);

/*
 * fa_paged_decode — one decode step over a paged KV cache ("Atención tipo
 * FlashAttention y atención paginada": a block table links logical positions to
 * fixed-size physical blocks, and the kernel translates every position through it).
 *   q [R,Hq,d] bf16: one new query token per request.
 *   k_cache, v_cache [num_blocks, Hkv, block_size, d] bf16.
 *   block_table [R, max_blocks_per_seq] int32: logical block -> physical block.
 *     Entries at or past ceil(ctx_lens[r] / block_size) are never read.
 *   ctx_lens [R] int32 (device): cached tokens of request r, 1 <= ctx <=
 *     max_blocks_per_seq * block_size.  The query attends to all of them.
 *   o [R,Hq,d] bf16.  lse [R,Hq] fp32 or NULL.
 *   d == 128, block_size == 16.
 *   A physical block id outside [0, num_blocks) or a ctx_len out of range is not
 *   dereferenced: the kernel skips it and sets the device status word
 *   (FA_ERR_INVALID_ARG), so the result for that request is undefined.
 *   Work split: each request's blocks are cut into splits of a fixed number of blocks
 *   (fa_set_decode_split), one CTA per (split, key/value head, request); splits of one
 *   request are merged by their lse weights.  The result does not depend on the split
 *   size beyond fp32 rounding order.
 *   If a bounded in-kernel wait runs out (fa_device_status then reports
 *   FA_ERR_DEVICE_TIMEOUT), o and lse of the affected requests are undefined (the
 *   kernels write NaN there rather than leftover partial results).
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE.
 */
fa_status fa_paged_decode(const void* q, const void* k_cache, const void* v_cache,
                          const int* block_table, const int* ctx_lens, void* o, float* lse,
                          int R, int Hq, int Hkv, int d, int block_size, int max_blocks_per_seq,
                          int num_blocks, float scale, fa_dtype dtype,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * fa_set_decode_split — number of cache blocks per split of fa_paged_decode (a multiple
 * of 4 in [32, 128]; 0 restores the library's default, 128 blocks = 2048 tokens at
 * block_size 16) for calls made after it, process-wide.  Smaller splits spread long
 * contexts over more CTAs at the cost of more partial results to merge.  The workspace
 * size depends on it: query fa_paged_decode_workspace_size after setting it.  Returns
 * the previous setting, or -1 (and changes nothing) for a value out of range.
 */
int fa_set_decode_split(int blocks);

/*
 * fa_paged_prefill — forward pass of a batch of variable-length sequences whose keys and
 * values sit in a paged KV cache ("Atención tipo FlashAttention y atención paginada": a
 * block table links logical positions to fixed-size physical blocks; the same page's
 * tiled online-softmax forward is run over the blocks the table names).
 *   Request r has ctx_lens[r] cached tokens (its keys and values, already written to the
 *   cache, e.g. by fa_paged_kv_append) and q_lens[r] query rows, which are the LAST
 *   q_lens[r] positions of its sequence (1 <= q_lens[r] <= ctx_lens[r]; equal for a
 *   fresh prompt, smaller for a chunk of a prompt whose earlier part is cached).
 *   q [R,Hq,Nq_max,d] bf16: query row i of request r at q[r,:,i,:], i < q_lens[r];
 *     q_lens[r] <= Nq_max.  Rows i >= q_lens[r] are not read into any result.
 *   k_cache, v_cache [num_blocks, Hkv, block_size, d] bf16; block_table [R,
 *     max_blocks_per_seq] int32 (entries at or past ceil(ctx_lens[r] / block_size) are
 *     never read); ctx_lens, q_lens [R] int32 (device).
 *   causal: 1 = query row i sees keys j <= i + ctx_lens[r] - q_lens[r] (its own position
 *     and every earlier one); 0 = it sees all ctx_lens[r] keys.
 *   o [R,Hq,Nq_max,d] bf16 and lse [R,Hq,Nq_max] fp32 (natural log): rows i >= q_lens[r]
 *     are left undefined (o) or untouched (lse).
 *   d in {64, 96, 128} (as fa_fwd), block_size == 16, GQA as in fa_fwd.
 *   A length or block id out of range is not dereferenced: the kernel skips that request
 *   (or reads block 0 for the bad entry) and sets the device status word
 *   (FA_ERR_INVALID_ARG), so that request's result is undefined.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA.
 */
fa_status fa_paged_prefill(const void* q, const void* k_cache, const void* v_cache,
                           const int* block_table, const int* ctx_lens, const int* q_lens,
                           void* o, float* lse, int R, int Hq, int Hkv, int Nq_max, int d,
                           int block_size, int max_blocks_per_seq, int num_blocks, float scale,
                           int causal, fa_dtype dtype, void* stream);

/*
 * fa_paged_kv_append — writes one new token per request into a paged KV cache ("Atención
 * tipo FlashAttention y atención paginada": the cache grows one token at a time and the
 * block table links logical positions to fixed-size physical blocks).
 *   k_new, v_new [R, Hkv, d] bf16: the new token's key and value for every KV head.
 *   positions [R] int32 (device): logical position of the new token in request r
 *     (its context length before the append); it goes to physical block
 *     block_table[r][pos / block_size], slot pos % block_size.
 *   k_cache, v_cache [num_blocks, Hkv, block_size, d] bf16, updated in place;
 *   block_table [R, max_blocks_per_seq] int32.
 *   d == 128, block_size == 16.  A position outside [0, max_blocks_per_seq*block_size)
 *   or a physical block outside [0, num_blocks) is not written; the kernel sets the
 *   device status word (FA_ERR_INVALID_ARG) instead.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED.
 */
fa_status fa_paged_kv_append(const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                             const int* block_table, const int* positions, int R, int Hkv, int d,
                             int block_size, int max_blocks_per_seq, int num_blocks, fa_dtype dtype,
                             void* stream);

/*
 * fa_paged_decode_noalloc — fa_paged_decode for callers that cannot allocate device
 * memory.  (No counterpart on the pages: this is a deployment variant of the decode
 * step, not part of the method.)
 *
 * Who needs it: code hosted inside a framework that owns all device allocations and
 * gives its kernels no workspace, and latency-critical loops that must not call
 * cudaMalloc after start-up (it can synchronise the device and take unbounded time).
 *
 * Arguments and results are those of fa_paged_decode minus the workspace: the split-KV
 * partials go to a fixed scratch array compiled into the library, FA_NOALLOC_SCRATCH_BYTES
 * (8 MiB) on every GPU that loads the library, held until the process exits.  Calls
 * whose fa_paged_decode_workspace_size(R, Hq, d, max_blocks_per_seq, block_size) exceeds
 * that limit are rejected with FA_ERR_WORKSPACE before anything is launched.  The
 * function never calls cudaMalloc, cudaFree or any allocating library routine.
 *
 * The first call on a device (with that device current) looks up the scratch array's
 * device address and caches it; make that first call before any stream capture.  The
 * cache is per CUDA context: after the device's context is destroyed and re-created
 * (cudaDeviceReset), the next call looks the address up again, so that call too should
 * come before any capture.  Every
 * call shares the one array, which keeps the last call's contents; nothing in it has to
 * start at zero (each partial the merge reads is written earlier in the same call).
 * Calls that overlap on the GPU (different streams, or different host threads without
 * ordering between them) race on the array and give undefined results.
 */
#define FA_NOALLOC_SCRATCH_BYTES (8u * 1024u * 1024u)
fa_status fa_paged_decode_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                  const int* block_table, const int* ctx_lens, void* o, float* lse,
                                  int R, int Hq, int Hkv, int d, int block_size, int max_blocks_per_seq,
                                  int num_blocks, float scale, fa_dtype dtype, void* stream);

/*
 * The passes around attention below take their arguments in one struct (read on the host during
 * the call): the fields that the comments name, pointers as everywhere, dtypes as fa_dtype.
 */

/*
 * Norm and rotation of q and k — the pass before attention (no counterpart on the pages).
 * Per head row x [d] with weight w [d] and n_axes positions per token:
 *   r = (mean_c x_c^2 + eps)^(-1/2),  y = x r w;  without weights y = x,
 *   each pair (a, b) of y turns by its angle t = positions[axis] * inv_freq[i]:
 *   a' = a cos t - b sin t,  b' = a sin t + b cos t.
 * Pair i of the rotary_dim / 2 pairs is (i, i + rotary_dim / 2), or (2i, 2i + 1) where
 * interleaved is 1; values at and past rotary_dim do not turn.  The first sections[0] pairs
 * follow axis 0 (time), the next sections[1] axis 1 (height), the last sections[2] axis 2
 * (width); the n_axes sections (1 to 3) sum to rotary_dim / 2.  Any int32 position
 * is exact: the angle is reduced in 64 bits.  Products, sums and the norm are fp32, rounded
 * once at the end.
 *
 * Common arguments:
 *   q_strides, k_strides (, v_strides): {batch, head, token} in elements, multiples
 *     of 16 bytes, so that views of a fused projection [B, N, heads, d] are read in place; a
 *     head's d values are contiguous.  0 repeats a row.
 *   q_weight, k_weight [d] of dtype `dtype`, or both NULL: no norm, the rotation alone.
 *   positions int32: axis a, batch b, token n at a * pos_axis_stride + b * pos_batch_stride + n
 *     (elements; a batch stride of 0 shares the positions).  inv_freq [rotary_dim / 2] double:
 *     radians per position.
 *   d in {64, 96, 128, 256}; rotary_dim a multiple of 16, at most d; eps > 0.
 *   Outputs may not overlap inputs.
 */

/*
 * fa_qk_norm_rope — q_out [B,Hq,N,d], k_out [B,Hkv,N,d] contiguous, as fa_fwd reads them; all
 * of dtype `dtype` (F32 or BF16).
 * Errors: FA_ERR_INVALID_ARG (null or misaligned pointer, bad size, stride, section, flag or
 * eps, one weight without the other); FA_ERR_UNSUPPORTED (other d, rotary_dim or dtype).
 */
typedef struct {
  const void *q, *k, *q_weight, *k_weight;
  const int* positions;
  const double* inv_freq;
  void *q_out, *k_out;
  int64_t q_strides[3], k_strides[3], pos_axis_stride, pos_batch_stride;
  int B, Hq, Hkv, N, d, rotary_dim, sections[3], n_axes, interleaved;
  float eps;
  int dtype;
} fa_qk_norm_rope_args;
fa_status fa_qk_norm_rope(const fa_qk_norm_rope_args* args, void* stream);

/*
 * fa_qk_norm_rope_append — the serving form: the same on R requests, with k' and v written
 * straight into the paged cache.  Lengths as in fa_paged_prefill: request r's tokens are the last
 * q_lens[r] positions of its ctx_lens[r] cached ones (0 <= q_lens[r] <= min(Nq_max, ctx_lens[r])),
 * so token i goes to cache position ctx_lens[r] - q_lens[r] + i; a decode step has Nq_max = 1 and
 * q_lens 1 (0: nothing to do for that request).  `positions` are the rotary ones: they need not
 * be cache positions (after an eviction they are not).
 *   q [R,Hq,Nq_max,d], k, v [R,Hkv,Nq_max,d] by strides, bf16; q_out [R,Hq,Nq_max,d] contiguous
 *   (the q of fa_paged_prefill, and for Nq_max = 1 that of the decode calls).  Rows i >=
 *   q_lens[r] are neither read nor written.
 *   k_cache, v_cache [num_blocks,Hkv,block_size,d], block_table [R,max_blocks_per_seq], ctx_lens,
 *   q_lens [R] int32 (device).  d in {64, 96, 128}, block_size == 16, dtype BF16.
 *   A length out of range skips the request, a block id out of range skips the token's cache
 *   write; either sets the device status word (FA_ERR_INVALID_ARG).  No two tokens of a call may
 *   share a cache slot.
 */
typedef struct {
  const void *q, *k, *v, *q_weight, *k_weight;
  const int* positions;
  const double* inv_freq;
  void *k_cache, *v_cache;
  const int *block_table, *ctx_lens, *q_lens;
  void* q_out;
  int64_t q_strides[3], k_strides[3], v_strides[3], pos_axis_stride, pos_batch_stride;
  int R, Hq, Hkv, Nq_max, d, block_size, max_blocks_per_seq, num_blocks, rotary_dim, sections[3], n_axes, interleaved;
  float eps;
  int dtype;
} fa_qk_norm_rope_append_args;
fa_status fa_qk_norm_rope_append(const fa_qk_norm_rope_append_args* args, void* stream);

/* fa_qk_norm_rope_bwd_workspace_size — bytes of device workspace fa_qk_norm_rope_bwd needs for its
 * partial weight gradients (none without weights).  Returns 0 for an invalid d. */
size_t fa_qk_norm_rope_bwd_workspace_size(int d);

/*
 * fa_qk_norm_rope_bwd — gradients of fa_qk_norm_rope, recomputing the norm from q and k.
 *   dq_out [B,Hq,N,d], dk_out [B,Hkv,N,d] contiguous, of dtype dout_dtype (what fa_bwd writes).
 *   q, k by strides, of dtype `dtype` (not read without weights).
 *   dq, dk of dtype grad_dtype by dq_strides, dk_strides (the projection's layout, for example);
 *   no two of its rows may share memory: each dimension larger than 1 has to step past all that the
 *   dimensions of smaller strides cover, as in any permuted slice of a dense array.
 *   dq_weight, dk_weight [d] fp32: the sums over every row of q, of k (with weights only).  The
 *   order of each sum is fixed: the same call gives the same bits.
 *   dtype BF16: dout_dtype and grad_dtype each F32 or BF16.  dtype F32: both F32.
 *   workspace: at least fa_qk_norm_rope_bwd_workspace_size(d) bytes, 256-byte aligned.
 * Errors: as fa_qk_norm_rope, plus FA_ERR_WORKSPACE.
 */
typedef struct {
  const void *dq_out, *dk_out, *q, *k, *q_weight, *k_weight;
  const int* positions;
  const double* inv_freq;
  void *dq, *dk;
  float *dq_weight, *dk_weight;
  void* workspace;
  size_t workspace_bytes;
  int64_t q_strides[3], k_strides[3], dq_strides[3], dk_strides[3], pos_axis_stride, pos_batch_stride;
  int B, Hq, Hkv, N, d, rotary_dim, sections[3], n_axes, interleaved;
  float eps;
  int dtype, dout_dtype, grad_dtype;
} fa_qk_norm_rope_bwd_args;
fa_status fa_qk_norm_rope_bwd(const fa_qk_norm_rope_bwd_args* args, void* stream);

/* fa_paged_decode_shared_workspace_size — bytes of device workspace fa_paged_decode_shared needs
 * for its partial results.  Returns 0 for invalid sizes. */
size_t fa_paged_decode_shared_workspace_size(int R, int Hq, int Hkv, int d, int max_prefix_blocks,
                                             int max_blocks_per_seq, int block_size);

/*
 * fa_paged_decode_shared — one decode step of R requests that share a prefix.  Request r attends
 * to the prefix's prefix_len[0] tokens and then to its own ctx_lens[r] ones; the prefix is read
 * and multiplied once for all requests, and the two partial results are merged by their mass.
 *   q [R,Hq,d] bf16; caches as in fa_paged_decode; prefix_table [max_prefix_blocks] and
 *   block_table [R,max_blocks_per_seq] int32; prefix_len [1], ctx_lens [R] int32 (device).
 *   Either length may be 0, up to its table's capacity; a request with no token at all gets
 *   o = 0 and lse = -inf.  Table entries past a length's last block are never read.
 *   o [R,Hq,d] bf16, lse [R,Hq] fp32 or NULL (natural log).  Weights enter the product with V to
 *   2^-16, whatever the batch and the tables' widths (these choose between two kernels, whose
 *   results may differ in the last bit of o).
 *   d in {64, 128}, block_size == 16, Hq / Hkv <= 16, dtype BF16; tables of up to 2^30 tokens (so
 *   in every call below, and in fa_qk_norm_rope_append).
 *   A length out of range or a bad block id is not dereferenced and sets the device status word
 *   (FA_ERR_INVALID_ARG); the results it belongs to are undefined.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE.
 */
typedef struct {
  const void *q, *k_cache, *v_cache;
  const int *prefix_table, *prefix_len, *block_table, *ctx_lens;
  void* o;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int R, Hq, Hkv, d, block_size, max_prefix_blocks, max_blocks_per_seq, num_blocks;
  float scale;
  int dtype;
} fa_paged_decode_shared_args;
fa_status fa_paged_decode_shared(const fa_paged_decode_shared_args* args, void* stream);

/* fa_paged_decode_scored_workspace_size — bytes of device workspace fa_paged_decode_scored needs
 * for its partial results and scores.  Returns 0 for invalid sizes. */
size_t fa_paged_decode_scored_workspace_size(int R, int Hq, int Hkv, int d, int max_blocks_per_seq, int block_size);

/*
 * fa_paged_decode_scored — a decode step (as fa_paged_decode; ctx_lens[r] may be 0: o = 0,
 * lse = -inf) that also adds up how much attention each cached token gets:
 *   weights[r, hkv, s] += sum over the query heads of hkv of e^{score_s - lse},  s < ctx_lens[r].
 *   weights [R, Hkv, max_blocks_per_seq * 16] fp32 by logical position, read and written; slots
 *   at and past ctx_lens[r] are left as they are.  Each slot is added to once, by one thread: the
 *   same call gives the same bits.
 *   d in {64, 128}, block_size == 16, Hq / Hkv <= 16, dtype BF16.
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE.
 */
typedef struct {
  const void *q, *k_cache, *v_cache;
  const int *block_table, *ctx_lens;
  float* weights;
  void* o;
  float* lse;
  void* workspace;
  size_t workspace_bytes;
  int R, Hq, Hkv, d, block_size, max_blocks_per_seq, num_blocks;
  float scale;
  int dtype;
} fa_paged_decode_scored_args;
fa_status fa_paged_decode_scored(const fa_paged_decode_scored_args* args, void* stream);

/* fa_paged_evict_workspace_size — bytes of device workspace fa_paged_evict needs for its lists of
 * moves.  Returns 0 where it needs none (few rows can move), and for invalid sizes. */
size_t fa_paged_evict_workspace_size(int R, int Hkv, int max_blocks_per_seq, int keep);

/*
 * fa_paged_evict — shrink each request's cache to `keep` tokens per kv head: the tokens among the
 * `recent` newest positions of its sequence, then the heaviest of the others by `weights` (ties:
 * the lower slot; -0 is 0, NaN lighter than anything).  0 <= recent <= keep, keep >= 1.  A request
 * with ctx_lens[r] <= keep loses nothing.
 *   Kept tokens in slots below `keep` stay; the i-th kept token at or past `keep` moves into the
 *   i-th freed slot below it, key and value (attention does not depend on the order of its keys;
 *   keys carry their rotation with them).  Each kv head keeps its own tokens.
 *   seq_lens [R] int32: tokens of the sequence so far, those evicted earlier among them
 *   (>= ctx_lens[r]).  slot_pos [R, Hkv, max_blocks_per_seq * 16] int32: the sequence position of
 *   the token in each slot, or negative for a slot filled by appending since the last eviction
 *   (its position is then seq_lens[r] - ctx_lens[r] + slot); start with -1 everywhere.
 *   weights as fa_paged_decode_scored keeps them.
 *   weights_out, slot_pos_out (same shapes, whole): each kept token's weight and position in its
 *   slot; 0 and -1 in every other slot, ready for tokens appended later.  new_ctx [R] =
 *   min(ctx_lens[r], keep).  They may not alias the inputs.
 *   k_cache, v_cache [num_blocks, Hkv, block_size, d] bf16, changed in place; a request's blocks
 *   must be its own (a shared prefix stays outside its block_table).
 *   d in {64, 96, 128, 256}, block_size == 16, dtype BF16.
 *   A length out of range leaves the request as it is, a block id out of range skips that move;
 *   either sets the device status word (FA_ERR_INVALID_ARG).
 * Errors: FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_WORKSPACE.
 */
typedef struct {
  void *k_cache, *v_cache;
  const int *block_table, *ctx_lens, *seq_lens;
  const float* weights;
  const int* slot_pos;
  float* weights_out;
  int *slot_pos_out, *new_ctx;
  void* workspace;
  size_t workspace_bytes;
  int R, Hkv, d, block_size, max_blocks_per_seq, num_blocks, keep, recent, dtype;
} fa_paged_evict_args;
fa_status fa_paged_evict(const fa_paged_evict_args* args, void* stream);

/*
 * fa_device_status — synchronises the current device and returns the device status
 * word the kernels set when a bounded wait runs out (FA_ERR_DEVICE_TIMEOUT) or a
 * block-table entry is out of range (FA_ERR_INVALID_ARG); FA_OK if none.  With
 * reset != 0 the word is cleared afterwards.
 */
fa_status fa_device_status(int reset);

/*
 * fa_set_wait_limit_ns — upper bound, in nanoseconds, on every in-kernel wait
 * launched after this call (default 2e8 ns = 200 ms).  Values < 1000 are clamped to 1000.
 */
void fa_set_wait_limit_ns(uint64_t ns);

/*
 * fa_selftest_wait_timeout — launches a one-CTA kernel that waits, with the current
 * limit, on a shared-memory barrier that nothing completes, so the wait must run
 * out.  Returns FA_OK if the launch succeeded; the kernel then sets the device status
 * word to FA_ERR_DEVICE_TIMEOUT, which fa_device_status reports.  For tests of the
 * timeout path; never faults or hangs the device.
 */
fa_status fa_selftest_wait_timeout(void* stream);

/*
 * fa_selftest_shared_timeout — fa_paged_decode_shared, whose prefix kernel loads no more than `tiles`
 * (>= 0) of a CTA's key tiles, so that the wait for the next one runs out after the current limit: the
 * rows behind it get NaN in o and lse, and the device status word FA_ERR_DEVICE_TIMEOUT.  For tests of
 * the timeout path, as above; FA_ERR_UNSUPPORTED for sizes that do not go to that kernel.
 */
fa_status fa_selftest_shared_timeout(const fa_paged_decode_shared_args* args, int tiles, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FA_H_ */
