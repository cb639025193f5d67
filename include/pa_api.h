/*
 * pa_api.h - C ABI of libpagedattn: attention over a paged KV cache on
 * NVIDIA GB300 (sm_103a).
 *
 * Two operations make up the path:
 *
 *   pa_write_kv   scatters each new token's K and V rows into its physical
 *                 cache slot through a slot mapping ("vLLM v1 Deep Dive: How
 *                 LLM(...) and the Server Boot and Generate", Part 3, "Aside -
 *                 KV cache and prefix caching": a slot is
 *                 block_id * block_size + offset and a scatter kernel writes
 *                 the freshly computed K/V there; "vLLM: An Exhaustive
 *                 Technical Study for Kernel Engineers", 2.1, "Reaching the
 *                 kernel").
 *
 *   pa_attention  runs attention for a unified mixed batch in one call:
 *                 prefill-chunk query spans attend causally over [their cached
 *                 prefix + their own new tokens], single-token decodes attend
 *                 over all of their blocks, every request reading K/V through
 *                 its own block table (same Aside, the block_table paragraph;
 *                 same page, Part 3, "Step 4c - Mixed batches" for
 *                 query_start_loc; "vLLM: An Exhaustive Technical Study for
 *                 Kernel Engineers", 2.4, "The seam" and "The backend
 *                 abstraction").
 *
 * Conventions shared by every call
 *  - All tensor arguments are DEVICE pointers owned by the caller. The library
 *    never allocates, frees or synchronises inside pa_write_kv/pa_attention;
 *    work is enqueued on `stream` (a cudaStream_t, or NULL for the legacy
 *    default stream) and the call returns at once.
 *  - Element type of q, k, v, k_cache, v_cache and out: bfloat16, passed as
 *    raw 16-bit storage. Index tensors: slot_mapping int64, the rest int32.
 *  - Layouts (row-major, contiguous):
 *      q, out            [num_tokens][num_q_heads][head_dim]
 *      k, v              [num_tokens][num_kv_heads][head_dim]
 *      k_cache, v_cache  [num_blocks][num_kv_heads][block_size][head_dim]
 *                        (one (block, kv head) is a contiguous block_size x
 *                        head_dim tile: the head-major "HND" block layout,
 *                        which "vLLM: An Exhaustive Technical Study for Kernel
 *                        Engineers", 2.6, names as the default for non-MLA
 *                        models)
 *      block_tables      [num_reqs][max_blocks_per_req]
 *      seq_lens          [num_reqs]
 *      query_start_loc   [num_reqs + 1], query_start_loc[0] == 0, non-decreasing
 *  - Supported shapes: block_size == 16; head_dim 64 or 128;
 *    num_q_heads / num_kv_heads (the GQA group) in {1, 2, 4, 8}. Other values
 *    return PA_ERR_UNSUPPORTED before anything is launched.
 *  - Every device pointer must be 16-byte aligned (PA_ERR_INVALID_ARG).
 *  - Errors that need the data to detect (a slot or block id outside the pool,
 *    seq_len shorter than the query span) are caught by the kernels: the bad
 *    item is skipped and a device error word is set, to be read with
 *    pa_get_device_error. Nothing traps and nothing waits unboundedly; a
 *    bounded wait that gives up reports PA_ERR_TIMEOUT the same way.
 *  - The first call on a device performs a one-time set-up (device property
 *    query and the address of the device error word); make one call, or
 *    pa_init, before capturing a stream into a CUDA graph.
 */
#ifndef PA_API_H
#define PA_API_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum pa_status {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = -1, /* null pointer, negative size, misaligned pointer, bad shape */
  PA_ERR_UNSUPPORTED = -2, /* block_size, head_dim or GQA group outside the supported set */
  PA_ERR_WORKSPACE = -3,   /* workspace null or smaller than pa_attention_workspace_size */
  PA_ERR_CUDA = -4,        /* a CUDA runtime call or a launch failed */
  PA_ERR_BOUNDS = -5,      /* (device error word) an index was outside its valid range */
  PA_ERR_TIMEOUT = -6      /* (device error word) a bounded wait in a kernel gave up */
} pa_status;

/* Device error word codes (pa_get_device_error `code`). */
#define PA_DEVERR_NONE 0
#define PA_DEVERR_SLOT 1         /* pa_write_kv: slot_mapping[t] >= num_blocks * block_size */
#define PA_DEVERR_BLOCK_ID 2     /* pa_attention: a block table entry outside [0, num_blocks) */
#define PA_DEVERR_LENGTHS 3      /* pa_attention: seq_len < query span, or too many blocks */
#define PA_DEVERR_QSL 4          /* pa_attention: query_start_loc not within [0, num_tokens] */
#define PA_DEVERR_WAIT_TIMEOUT 5 /* a kernel's bounded wait on a copy gave up */
#define PA_DEVERR_PREFIX 6       /* pa_attention_cascade: a request's table does not start
                                    with request 0's common-prefix blocks;
                                    pa_attention_shared: with its group's, or a
                                    group's prefix length is not one */
#define PA_DEVERR_POSITION 7     /* pa_norm_rope_write_kv: a position outside the table */

/*
 * One-time per-device set-up for the current device (see the conventions).
 * Idempotent; the other calls do it on first use.
 */
pa_status pa_init(void);

/*
 * Scatter new K/V rows into the paged caches.
 *   k, v           [num_tokens][num_kv_heads][head_dim] bf16, read only
 *   slot_mapping   [num_tokens] int64; token t goes to block
 *                  slot_mapping[t] / block_size, row slot_mapping[t] % block_size.
 *                  A negative slot marks a padding token: it is skipped.
 *   k_cache, v_cache  written at the named slots only; every other slot keeps
 *                  its contents, bit for bit.
 * Copies are exact (bit patterns). Two tokens naming the same slot is the
 * caller's error; which one lands is unspecified. A slot >= num_blocks *
 * block_size is skipped and sets PA_DEVERR_SLOT.
 * head_dim here may be any multiple of 8 (the scatter is type-agnostic).
 */
pa_status pa_write_kv(const void* k, const void* v, const int64_t* slot_mapping,
                      void* k_cache, void* v_cache, int num_tokens, int num_kv_heads,
                      int head_dim, int block_size, int num_blocks, void* stream);

/*
 * Bytes of device workspace pa_attention needs for a batch of this size
 * (planner output and split-KV partial results). The value
 * depends only on the arguments, not on the device. Returns 0 on bad
 * arguments.
 */
size_t pa_attention_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                   int num_kv_heads, int head_dim);

/*
 * Attention for a mixed batch of decodes and prefill chunks.
 *   q                [num_tokens][num_q_heads][head_dim] bf16
 *   k_cache, v_cache the pool, already holding this step's new K/V
 *                    (call pa_write_kv first, on the same stream)
 *   block_tables     request r's logical block i is physical block
 *                    block_tables[r][i]; entries past ceil(seq_lens[r] / 16)
 *                    are never read
 *   seq_lens         total KV length of each request, new tokens included
 *   query_start_loc  request r's new tokens are rows
 *                    query_start_loc[r] .. query_start_loc[r+1]-1 of q/out;
 *                    with qlen = that count and ctx = seq_lens[r] - qlen, row
 *                    j attends to keys 0 .. ctx + j (causal, bottom-right
 *                    aligned; a decode is qlen 1 and sees every key)
 *   scale            multiplies q.k before the softmax (usually 1/sqrt(head_dim))
 *   out              [num_tokens][num_q_heads][head_dim] bf16; rows of
 *                    requests with qlen 0 and rows past query_start_loc[num_reqs]
 *                    are left untouched. Device memory, or pinned host memory
 *                    through the address pa_mapped_pointer gives: the kernels
 *                    then store the result across the host link as they
 *                    finish it, so no separate device-to-host copy follows.
 *   query head h reads KV head h / (num_q_heads / num_kv_heads)
 *   max_blocks_per_req  row stride of block_tables
 *   max_query_len, max_seq_len  host-side upper bounds the scheduler already
 *                    knows; they only size launches (max_query_len <= 1 skips
 *                    the prefill-chunk kernel). Values below the true maxima
 *                    are an error (PA_DEVERR_LENGTHS).
 *   workspace        device buffer of at least
 *                    pa_attention_workspace_size(...) bytes, 256-byte aligned,
 *                    no initial contents required; it must not be used by
 *                    another call that runs concurrently on the GPU.
 */
pa_status pa_attention(const void* q, const void* k_cache, const void* v_cache,
                       const int32_t* block_tables, const int32_t* seq_lens,
                       const int32_t* query_start_loc, float scale, void* out, int num_reqs,
                       int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                       int block_size, int num_blocks, int max_blocks_per_req,
                       int max_query_len, int max_seq_len, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * FP8 KV cache ("vLLM: An Exhaustive Technical Study for Kernel Engineers",
 * 2.8 Quantization & compute kernels: --kv-cache-dtype fp8 stores K and V as
 * E4M3 with one fp32 scale per tensor, k_scale and v_scale; FP8 halves the
 * bytes of a block). E4M3 here is the OCP 8-bit format the GPU implements:
 * 1 sign, 4 exponent bits (bias 7), 3 mantissa bits, no infinities, largest
 * finite 448.
 *
 * pa_write_kv_fp8: as pa_write_kv, but the caches hold one byte per element
 * ([num_blocks][num_kv_heads][block_size][head_dim] uint8) and each element
 * is stored as E4M3(x / scale): the quotient is a correctly rounded binary32
 * division, the conversion rounds to nearest even and saturates at +-448.
 * k_scale / v_scale must be finite and > 0 (PA_ERR_INVALID_ARG otherwise).
 */
pa_status pa_write_kv_fp8(const void* k, const void* v, const int64_t* slot_mapping,
                          void* k_cache, void* v_cache, float k_scale, float v_scale,
                          int num_tokens, int num_kv_heads, int head_dim, int block_size,
                          int num_blocks, void* stream);

/*
 * pa_attention_fp8: pa_attention over E4M3 caches written by pa_write_kv_fp8.
 * Keys are value(code) * k_scale and values value(code) * v_scale, and the
 * dequantisation is fused into both attention kernels, as for a bf16 cache:
 *  - prefill chunks (spans of 16 or more new tokens) run on the tensor-core
 *    kernel, whose converter warps widen each E4M3 tile exactly to bf16 in
 *    shared memory before the bf16 MMA;
 *  - every other span (decodes, short spans) runs on the CUDA-core split-KV
 *    kernel, which widens codes exactly to fp32.
 * k_scale is folded into the query scaling and v_scale into the output. The
 * workspace is pa_attention_workspace_size(...) bytes, as for pa_attention.
 * Errors as pa_attention, plus PA_ERR_INVALID_ARG for a scale that is not
 * finite and > 0.
 */
pa_status pa_attention_fp8(const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* seq_lens,
                           const int32_t* query_start_loc, float scale, float k_scale,
                           float v_scale, void* out, int num_reqs, int num_tokens,
                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           int num_blocks, int max_blocks_per_req, int max_query_len,
                           int max_seq_len, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Per-head norm, position rotation and KV-cache write in one pass: what a
 * decoder layer does with its projections before attention. The scatter is
 * pa_write_kv's ("vLLM v1 Deep Dive: How LLM(...) and the Server Boot and
 * Generate", Part 3, "Aside - KV cache and prefix caching"); the norm and the
 * rotation in front of it are the pages' "model" side and have no counterpart
 * there.
 *   q  [num_tokens][num_q_heads][head_dim], k, v [num_tokens][num_kv_heads]
 *      [head_dim], bf16. A token's heads are contiguous; tokens are q_stride /
 *      k_stride / v_stride elements apart (at least one token's heads, a
 *      multiple of 8), so the three may be parts of one projection's output.
 *   q_weight, k_weight  [head_dim] bf16, or NULL: that kind of head is not
 *      normalised. y = x * w / sqrt(mean(x^2) + eps); eps finite and >= 0.
 *   positions, cos_sin  positions[t] (int32) picks row cos_sin[positions[t]]
 *      of the table [max_position][rotary_dim] fp32: the rotary_dim / 2
 *      cosines, then the sines. rotary_dim is a multiple of 16 up to head_dim;
 *      0 turns the rotation off (positions and cos_sin may then be NULL).
 *   interleaved  0: elements i and i + rotary_dim / 2 are a pair; else 2i and
 *      2i + 1. Elements past rotary_dim keep their value.
 *   q_out  [num_tokens][num_q_heads][head_dim] bf16, contiguous; it may be q
 *      itself where q is contiguous, and overlaps no other argument.
 *   k_cache, v_cache, slot_mapping  as for pa_write_kv. A negative slot marks
 *      a padding token, of which nothing is written, q_out included.
 * Arithmetic is binary32, each result rounded once. head_dim 64 or 128, up to
 * 65536 heads of a kind. A slot outside the pool sets PA_DEVERR_SLOT and a position
 * outside the table PA_DEVERR_POSITION; such a token is skipped whole.
 */
pa_status pa_norm_rope_write_kv(const void* q, const void* k, const void* v, long long q_stride,
                                long long k_stride, long long v_stride, const int32_t* positions,
                                const float* cos_sin, const void* q_weight, const void* k_weight,
                                float eps, int rotary_dim, int interleaved, int max_position,
                                const int64_t* slot_mapping, void* q_out, void* k_cache,
                                void* v_cache, int num_tokens, int num_q_heads, int num_kv_heads,
                                int head_dim, int block_size, int num_blocks, void* stream);

/* The same into E4M3 caches: each element of K and V is stored as
 * E4M3(y / scale), as pa_write_kv_fp8 does, from the binary32 y. */
pa_status pa_norm_rope_write_kv_fp8(const void* q, const void* k, const void* v,
                                    long long q_stride, long long k_stride, long long v_stride,
                                    const int32_t* positions, const float* cos_sin,
                                    const void* q_weight, const void* k_weight, float eps,
                                    int rotary_dim, int interleaved, int max_position,
                                    const int64_t* slot_mapping, void* q_out, void* k_cache,
                                    void* v_cache, float k_scale, float v_scale, int num_tokens,
                                    int num_q_heads, int num_kv_heads, int head_dim,
                                    int block_size, int num_blocks, void* stream);

/*
 * Cascade attention for a batch whose requests all share one common prefix
 * ("vLLM: An Exhaustive Technical Study for Kernel Engineers", 2.3 Automatic
 * prefix caching & KV reuse, cascade attention: when every request of a batch
 * shares one prefix, attention over the prefix is computed once for the whole
 * batch and merged with each request's attention over its own suffix by
 * log-sum-exp renormalisation; metadata common_prefix_len).
 *
 * The result equals pa_attention's on the same arguments (up to fp32 rounding
 * order). Arguments are pa_attention's plus:
 *   common_prefix_len  tokens of the shared prefix: a positive multiple of
 *                      block_size. Every request's first common_prefix_len /
 *                      block_size block-table entries must equal request 0's,
 *                      and every request's context (seq_len minus its new
 *                      tokens) must be at least common_prefix_len, so that
 *                      each new token sees the whole prefix.
 *   workspace          at least pa_attention_cascade_workspace_size(...) bytes.
 * The prefix pass runs on the tensor cores: for each KV head, the prefix keys
 * against the queries of every new token of the batch (all G heads), split
 * over key chunks, giving fp32 partials (max, sum, unnormalised output) in
 * the workspace. The split-KV kernel then attends each token to its own
 * suffix keys only and folds the prefix partials into its merge. Every span
 * is handled by the split-KV kernel (no prefill-chunk tiles).
 * Errors: host-side as pa_attention, plus PA_ERR_INVALID_ARG for a
 * common_prefix_len that is not a positive multiple of block_size. On the
 * device, a request whose context is shorter than the prefix sets
 * PA_DEVERR_LENGTHS and is skipped (its rows untouched); a request whose
 * table does not start with request 0's prefix blocks sets PA_DEVERR_PREFIX,
 * and its rows are computed with request 0's prefix (they are wrong; the
 * error word says so).
 */
size_t pa_attention_cascade_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim);

pa_status pa_attention_cascade(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               const int32_t* query_start_loc, float scale, void* out,
                               int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks,
                               int max_blocks_per_req, int max_query_len, int max_seq_len,
                               int common_prefix_len, void* workspace, size_t workspace_bytes,
                               void* stream);

/*
 * Attention with a sliding window and visible first tokens: pa_attention where
 * a new token at position p (its request's context plus its place in the span)
 * attends to keys i <= p with i > p - window or i < sinks, i.e. to the last
 * `window` keys, its own included, and the first `sinks`. The pages name
 * sliding-window layers ("vLLM: An Exhaustive Technical Study for Kernel
 * Engineers", 2.1, hybrid KV cache groups) and sinks (2.4, the TRT-LLM
 * backend) without describing either.
 *   window >= 1, sinks >= 0 (PA_ERR_INVALID_ARG). A window of max_seq_len keys
 *   or more is pa_attention, bit for bit.
 * The other arguments, the workspace and the errors are pa_attention's (_fp8:
 * pa_attention_fp8's). The tables keep their logical layout, so a request's
 * blocks that none of its new tokens attends to may have been released: their
 * table entries are not read, whatever they hold. Of the keys in a block that
 * is read, those that no new token of the request attends to may hold
 * anything; K and V of the others must be finite, as for pa_attention. Time
 * and bytes follow the keys attended to, not the sequence length. num_blocks
 * >= 1. Where the tensor cores take the products (prompt chunks; decodes by
 * PA_OPT_DECODE_TC) the softmax weights are rounded to bf16 for them, or over an
 * E4M3 cache's decodes to two E4M3 terms each, as in pa_attention: an output is
 * within 2^-7 of its weights' sum of |V|, and its own rounding.
 */
pa_status pa_attention_window(const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* block_tables, const int32_t* seq_lens,
                              const int32_t* query_start_loc, float scale, void* out,
                              int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                              int head_dim, int block_size, int num_blocks,
                              int max_blocks_per_req, int max_query_len, int max_seq_len,
                              int window, int sinks, void* workspace, size_t workspace_bytes,
                              void* stream);

pa_status pa_attention_window_fp8(const void* q, const void* k_cache, const void* v_cache,
                                  const int32_t* block_tables, const int32_t* seq_lens,
                                  const int32_t* query_start_loc, float scale, float k_scale,
                                  float v_scale, void* out, int num_reqs, int num_tokens,
                                  int num_q_heads, int num_kv_heads, int head_dim,
                                  int block_size, int num_blocks, int max_blocks_per_req,
                                  int max_query_len, int max_seq_len, int window, int sinks,
                                  void* workspace, size_t workspace_bytes, void* stream);

/*
 * Accumulated attention weight of every cached key: what pa_evict_kv goes by.
 * The pages have no counterpart.
 *   out[r][h][i] = (i < ctx ? weights[r][h][i] : 0) + sum over the request's
 *                  new tokens and the G query heads of KV head h of the softmax
 *                  weight pa_attention gives key i
 * with ctx = seq_lens[r] minus the new tokens, for 0 <= i < seq_lens[r]; a key
 * that is new in this step starts at zero, so a fresh request's row needs no
 * clearing. Entries past seq_lens[r], and the rows of requests without new
 * tokens, are left untouched. Call it on the arguments of pa_attention, before
 * or after it.
 *   weights, out  [num_reqs][num_kv_heads][weights_stride] fp32; out may be
 *                 weights itself (accumulation in place), else they must not
 *                 overlap
 *   workspace     at least pa_attention_weights_workspace_size(...) bytes,
 *                 256-byte aligned, no initial contents required, used by one
 *                 call at a time. The size grows with num_reqs x max_seq_len:
 *                 4 bytes per (request, query head, key) for a decode batch.
 * The other arguments are pa_attention's, and so are the limits (head_dim 64 or
 * 128, groups of 1, 2, 4 or 8; num_blocks >= 1) and the errors. A request longer than
 * weights_stride sets PA_DEVERR_LENGTHS and is skipped. Scores and sums are
 * binary32; results do not depend on the order in which CTAs run. In spans of
 * more than 8 rows (tokens x G) so is a row's log-sum-exp, whose rounding its
 * weights take over: a relative error of |lse| x 2^-24, so scores there should
 * stay below some 10^4. A NaN or an infinity in a query or in a key makes NaN
 * of the weights of every key that the row, or a row that sees the key, sees.
 */
size_t pa_attention_weights_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                           int num_kv_heads, int head_dim, int max_query_len,
                                           int max_seq_len);

pa_status pa_attention_weights(const void* q, const void* k_cache, const int32_t* block_tables,
                               const int32_t* seq_lens, const int32_t* query_start_loc,
                               float scale, const float* weights, float* out,
                               long long weights_stride, int num_reqs, int num_tokens,
                               int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                               int num_blocks, int max_blocks_per_req, int max_query_len,
                               int max_seq_len, void* workspace, size_t workspace_bytes,
                               void* stream);

/* The same over an E4M3 key cache (keys are value(code) * k_scale). */
pa_status pa_attention_weights_fp8(const void* q, const void* k_cache,
                                   const int32_t* block_tables, const int32_t* seq_lens,
                                   const int32_t* query_start_loc, float scale, float k_scale,
                                   const float* weights, float* out, long long weights_stride,
                                   int num_reqs, int num_tokens, int num_q_heads,
                                   int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                   int max_blocks_per_req, int max_query_len, int max_seq_len,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Cut a cache to `keep` tokens per KV head by accumulated attention weight.
 * The pages leave eviction at the block level ("Inside the vLLM Engine", "The
 * pool, the queue, and the hash"); this one drops tokens of a live request.
 *
 * Every request r with seq_lens[r] > keep is cut: each of its KV heads keeps
 * the first `sinks` tokens, the last `recent` ones, and of the tokens between
 * them the keep - sinks - recent with the largest weights (equal weights: the
 * lowest position; a NaN counts less than any number). Their K and V rows are
 * copied, in order of position, to the blocks new_block_tables[r]: the n-th
 * kept token of a head to row n % 16 of block new_block_tables[r][n / 16].
 * Rows past `keep` of the last new block are left untouched, and so are the
 * old blocks. The heads of a request choose separately, so a slot no longer
 * holds one token in all heads; attention does not need it to. Keys are moved
 * as they are: a rotation by position stays the one they were written with.
 * Requests with seq_lens[r] <= keep are left as they are: only new_seq_lens[r]
 * is written for them.
 *   k_cache, v_cache  the pool, elem_bytes (2: bf16, 1: E4M3 codes with a scale per
 *                     tensor) per element; a row-scaled cache's scales are not moved
 *   weights           [num_reqs][num_kv_heads][weights_stride] fp32, entries
 *                     past a request's length not read (pa_attention_weights
 *                     makes them)
 *   new_block_tables  [num_reqs][max_new_blocks], max_new_blocks >=
 *                     ceil(keep / 16). The blocks named for the requests that
 *                     are cut must be distinct, and none of them may be a block
 *                     that a request still holds: the copy is out of place.
 *   new_seq_lens      [num_reqs] int32: min(seq_lens[r], keep); not seq_lens itself
 *   kept              [num_reqs][num_kv_heads][keep] int32: the positions kept,
 *                     rising (written for the requests that are cut)
 *   new_weights       [num_reqs][num_kv_heads][new_weights_stride] fp32 or
 *                     NULL: the kept tokens' weights; it must not overlap weights
 *   max_seq_len       upper bound of seq_lens; a longer request, or one that
 *                     its table or weights do not hold, sets PA_DEVERR_LENGTHS
 *                     and is skipped
 * sinks, recent >= 0, keep >= 1, sinks + recent <= keep (PA_ERR_INVALID_ARG).
 * head_dim 64 or 128, block_size 16. A block id outside the pool sets
 * PA_DEVERR_BLOCK_ID and its rows are not copied.
 */
pa_status pa_evict_kv(void* k_cache, void* v_cache, const int32_t* block_tables,
                      const int32_t* seq_lens, const float* weights,
                      const int32_t* new_block_tables, int32_t* new_seq_lens, int32_t* kept,
                      float* new_weights, int num_reqs, int num_kv_heads, int head_dim,
                      int elem_bytes, int block_size, int num_blocks, int max_blocks_per_req,
                      int max_new_blocks, long long weights_stride, long long new_weights_stride,
                      int max_seq_len, int keep, int recent, int sinks, void* stream);

/*
 * pa_attention without a caller-provided workspace, for callers that cannot
 * allocate device memory (for example code running inside an allocator's own
 * callbacks, or under a host framework that owns all device memory and offers
 * no allocation hook). The pages describe no such entry point; it has no
 * counterpart there.
 *
 * Arguments are those of pa_attention minus workspace / workspace_bytes; the
 * caller still passes every input and output. The workspace is a fixed
 * scratch array of PA_NOALLOC_SCRATCH_BYTES compiled into the library: each
 * GPU that loads the library holds it until the process exits. The call
 * allocates nothing (no cudaMalloc, no cudaFree, no library allocator).
 *  - A batch whose pa_attention_workspace_size(...) exceeds
 *    PA_NOALLOC_SCRATCH_BYTES is rejected with PA_ERR_WORKSPACE before
 *    anything is launched.
 *  - Argument errors are reported as pa_attention reports them (the same
 *    codes, checked first), whatever the batch size; the size check follows.
 *  - The first call on a device looks up the scratch array's device address
 *    (with that device current). With lazy module loading (the CUDA default)
 *    that lookup is also when the driver places the array in device memory:
 *    an allocation the driver makes once, on that first call. So make the
 *    first call on each device outside any context that must not allocate,
 *    and before any stream capture; later calls allocate nothing.
 *  - Every call on a device shares the one scratch array, which keeps the
 *    last call's contents; the kernels re-initialise everything they read
 *    from it on each call. Calls whose work overlaps on the GPU (different
 *    streams, or different host threads without ordering) race on the
 *    scratch and give wrong results: serialise them.
 */
#define PA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

pa_status pa_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                               const int32_t* block_tables, const int32_t* seq_lens,
                               const int32_t* query_start_loc, float scale, void* out,
                               int num_reqs, int num_tokens, int num_q_heads, int num_kv_heads,
                               int head_dim, int block_size, int num_blocks,
                               int max_blocks_per_req, int max_query_len, int max_seq_len,
                               void* stream);

/*
 * The calls above with many arguments, taking them in a struct: for bindings
 * that pay per argument (a foreign-function layer spends longer converting
 * twenty-five arguments than a small kernel runs). kv_fp8 selects the _fp8
 * form and its scales, which are ignored otherwise; pa_evict_kv has none. The
 * results and errors are those of the calls they stand for; args == NULL is
 * PA_ERR_INVALID_ARG. The structs hold pointers first, then 64-bit, then
 * 32-bit members, without padding but for the end; pa_args_size(i) is the
 * size of the i-th struct below, for a binding to check its layout against
 * (0 for another i).
 */
typedef struct pa_norm_rope_write_args { /* 0 */
  const void *q, *k, *v;
  const int32_t* positions;
  const float* cos_sin;
  const void *q_weight, *k_weight;
  const int64_t* slot_mapping;
  void *q_out, *k_cache, *v_cache, *stream;
  long long q_stride, k_stride, v_stride;
  float eps, k_scale, v_scale;
  int rotary_dim, interleaved, max_position, kv_fp8;
  int num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
} pa_norm_rope_write_args;
pa_status pa_norm_rope_write_kv_args(const pa_norm_rope_write_args* args);

typedef struct pa_window_args { /* 1 */
  const void *q, *k_cache, *v_cache;
  const int32_t *block_tables, *seq_lens, *query_start_loc;
  void *out, *workspace, *stream;
  size_t workspace_bytes;
  float scale, k_scale, v_scale;
  int kv_fp8, num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
  int max_blocks_per_req, max_query_len, max_seq_len, window, sinks;
} pa_window_args;
pa_status pa_attention_window_args(const pa_window_args* args);

typedef struct pa_weights_args { /* 2 */
  const void *q, *k_cache;
  const int32_t *block_tables, *seq_lens, *query_start_loc;
  const float* weights;
  float* out;
  void *workspace, *stream;
  size_t workspace_bytes;
  long long weights_stride;
  float scale, k_scale;
  int kv_fp8, num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
  int max_blocks_per_req, max_query_len, max_seq_len;
} pa_weights_args;
pa_status pa_attention_weights_args(const pa_weights_args* args);

typedef struct pa_evict_args { /* 3 */
  void *k_cache, *v_cache;
  const int32_t *block_tables, *seq_lens;
  const float* weights;
  const int32_t* new_block_tables;
  int32_t *new_seq_lens, *kept;
  float* new_weights;
  void* stream;
  long long weights_stride, new_weights_stride;
  int num_reqs, num_kv_heads, head_dim, elem_bytes, block_size, num_blocks;
  int max_blocks_per_req, max_new_blocks, max_seq_len, keep, recent, sinks;
} pa_evict_args;
pa_status pa_evict_kv_args(const pa_evict_args* args);

size_t pa_args_size(int which);

/*
 * Row-scaled E4M3 caches: K and V as E4M3 codes with one power of two for every
 * row (the head_dim elements of one token and KV head), which the write finds.
 * The pages' FP8 cache has one scale per tensor, to be known before the first
 * write; they have no counterpart to this one.
 *   k_cache, v_cache  [num_blocks][num_kv_heads][16][head_dim] codes, as for
 *                     pa_write_kv_fp8
 *   scales            [num_blocks][num_kv_heads][2][16] bytes, 16-byte aligned:
 *                     K's 16 rows of a block, then V's. A byte b stands for
 *                     2^(b - 127) (the 8-bit format with an exponent only),
 *                     255 for NaN.
 * With a the largest |x| of a row, e is the smallest integer of [-100, 119] with
 * a <= 448 x 2^e, b = e + 127, and an element's code is E4M3(x 2^-e), rounded
 * once, to nearest even, saturating at +-448 (which only rows past 448 x 2^119
 * reach). A row's value is code x 2^e, a bf16 number. A row with an infinity or
 * a NaN gets b = 255 and codes of zero, and reads back as NaN. The calls that
 * read such a cache take the bytes that these writes make (27 to 246, 255).
 *
 * The calls from here on take their arguments in a struct only, laid out like the
 * structs above; pa_args_size(16 + i) is the size of the i-th. NULL is
 * PA_ERR_INVALID_ARG.
 */

/* pa_write_kv into a row-scaled cache. Tokens of k and v are k_stride / v_stride
 * elements apart (at least one token's heads, a multiple of 8), a token's heads
 * contiguous. head_dim 64 or 128, up to 65536 KV heads; a negative slot is
 * skipped, one outside the pool too, with PA_DEVERR_SLOT. The other slots of a call
 * are distinct: of tokens with the same one, a row may keep one's codes and another's
 * scale. */
typedef struct pa_write_rows_args { /* 16 */
  const void *k, *v;
  const int64_t* slot_mapping;
  void *k_cache, *v_cache;
  uint8_t* scales;
  void* stream;
  long long k_stride, v_stride;
  int num_tokens, num_kv_heads, head_dim, block_size, num_blocks;
} pa_write_rows_args;
pa_status pa_write_kv_rows(const pa_write_rows_args* args);

/* pa_norm_rope_write_kv into a row-scaled cache: each row of K and V from the
 * binary32 values, its scale from theirs. */
typedef struct pa_norm_rope_write_rows_args { /* 17 */
  const void *q, *k, *v;
  const int32_t* positions;
  const float* cos_sin;
  const void *q_weight, *k_weight;
  const int64_t* slot_mapping;
  void *q_out, *k_cache, *v_cache;
  uint8_t* scales;
  void* stream;
  long long q_stride, k_stride, v_stride;
  float eps;
  int rotary_dim, interleaved, max_position;
  int num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
} pa_norm_rope_write_rows_args;
pa_status pa_norm_rope_write_kv_rows(const pa_norm_rope_write_rows_args* args);

/*
 * pa_attention over a row-scaled cache: keys are code x 2^e of their row, values
 * alike. Prompt chunks (spans of 16 or more new tokens) run on the tensor-core
 * kernel over tiles widened to bf16, exactly; every other span on a split-KV
 * kernel that takes a key's 2^e after the products with its codes and a value's
 * before. The workspace is pa_attention_workspace_size(...) bytes; limits and
 * errors are pa_attention's. A row that reads back as NaN makes NaN of the outputs
 * that attend to it, and in a prompt chunk may make NaN of those of earlier
 * tokens of the chunk, for the query heads of its KV head. V rows past 448 x 2^100
 * may lose the smaller keys' part.
 */
typedef struct pa_attention_rows_args { /* 18 */
  const void *q, *k_cache, *v_cache;
  const uint8_t* scales;
  const int32_t *block_tables, *seq_lens, *query_start_loc;
  void *out, *workspace, *stream;
  size_t workspace_bytes;
  float scale;
  int num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
  int max_blocks_per_req, max_query_len, max_seq_len;
} pa_attention_rows_args;
pa_status pa_attention_rows(const pa_attention_rows_args* args);

/*
 * Read ranges of cached keys and values back, dense and in bf16: for another
 * cache or format, or for code that knows no block tables. The pages have no
 * counterpart.
 *   read_start_loc  [num_reqs + 1] int32, non-decreasing: request r's keys go to
 *                   rows read_start_loc[r] .. read_start_loc[r + 1] - 1 of
 *                   k_out and v_out; rows of no request are left untouched
 *   first           [num_reqs] int32: the first key read, or NULL: key 0
 *   k_out, v_out    [num_tokens][num_kv_heads][head_dim] bf16, 32-byte aligned
 *   kv_format       0: bf16 caches, copied bit for bit; 1: E4M3 with k_scale and
 *                   v_scale, the binary32 product rounded once; 2: row-scaled
 *                   (scales), exact
 *   num_tokens      rows of k_out and v_out
 * head_dim 64 or 128, up to 8192 KV heads. Errors: a request whose rows do not lie
 * in [0, num_tokens] sets PA_DEVERR_QSL, one whose keys its table does not hold
 * PA_DEVERR_LENGTHS, and is skipped; a key whose block id is outside the pool sets
 * PA_DEVERR_BLOCK_ID and its row is left untouched.
 */
typedef struct pa_read_args { /* 19 */
  const void *k_cache, *v_cache;
  const uint8_t* scales;
  const int32_t *block_tables, *read_start_loc, *first;
  void *k_out, *v_out, *stream;
  float k_scale, v_scale;
  int kv_format, num_reqs, num_tokens, num_kv_heads, head_dim, block_size, num_blocks;
  int max_blocks_per_req;
} pa_read_args;
pa_status pa_read_kv(const pa_read_args* args);

/*
 * Attention for a batch whose requests share prefixes in groups, over any cache
 * format: pa_attention's result (up to the order of sums and the tolerances of
 * the kernels), with every group's prefix attended to once for all of its tokens.
 * The pages describe one prefix common to the whole batch ("vLLM: An Exhaustive
 * Technical Study for Kernel Engineers", 2.3, cascade attention; here
 * pa_attention_cascade) and fall back to plain attention for a forest of them.
 *   group_start_loc  [num_groups + 1] int32, non-decreasing: requests
 *                    group_start_loc[g] .. group_start_loc[g + 1] - 1 are group g;
 *                    requests before the first and behind the last share nothing
 *   prefix_lens      [num_groups] int32: tokens of the group's prefix, a multiple
 *                    of 16, at most max_prefix_len; 0: the group shares nothing.
 *                    The prefix's blocks start the tables of all of its requests.
 *   max_prefix_len   host-side upper bound; sizes the workspace
 *   kv_format, scales, k_scale, v_scale  as for pa_read_kv
 *   workspace        at least pa_attention_shared_workspace_size(...) bytes
 * The other arguments are pa_attention's. Sharing follows the lengths: a request
 * that does not see its whole prefix (a context shorter than it), that brings 16 or
 * more new tokens (a prompt chunk, whose rows share K and V already) or that is
 * left alone with one token attends on its own, with the same result; and so does the
 * whole batch where sharing would not pay (PA_OPT_SHARED_MIN_KB).
 * The prefixes run on the tensor cores as a cascade's does, in pairs of 128-row
 * tiles of a group's queries and chunks of keys, into fp32 partials; each token's
 * own keys on the split-KV kernels; a merge pass folds both. At most 1024 groups,
 * num_reqs x max_blocks_per_req below 2^31 (PA_ERR_UNSUPPORTED); num_blocks >= 1.
 * Errors: host-side as pa_attention. On the device, beside pa_attention's: a group
 * whose requests are not of the batch sets PA_DEVERR_QSL, one whose prefix is
 * negative, no multiple of 16 or longer than max_prefix_len PA_DEVERR_PREFIX (its
 * requests then attend on their own); a sharing request whose table does not start
 * with the blocks of the group's first sharing request sets PA_DEVERR_PREFIX, and
 * is computed with that one's prefix where the batch shares (the result is wrong; the
 * error word says so). With no groups, or max_prefix_len below 16, the call is
 * pa_attention's and reads neither group_start_loc nor prefix_lens.
 */
size_t pa_attention_shared_workspace_size(int num_reqs, int num_tokens, int num_q_heads,
                                          int num_kv_heads, int head_dim, int num_groups,
                                          int max_prefix_len);

typedef struct pa_shared_args { /* 20 */
  const void *q, *k_cache, *v_cache;
  const uint8_t* scales;
  const int32_t *block_tables, *seq_lens, *query_start_loc, *group_start_loc, *prefix_lens;
  void *out, *workspace, *stream;
  size_t workspace_bytes;
  float scale, k_scale, v_scale;
  int kv_format, num_reqs, num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks;
  int max_blocks_per_req, max_query_len, max_seq_len, num_groups, max_prefix_len;
} pa_shared_args;
pa_status pa_attention_shared(const pa_shared_args* args);

/* Size of the fixed scratch array used by pa_attention_noalloc. */
size_t pa_noalloc_scratch_bytes(void);

/* Human-readable name of a pa_status value (static string). */
const char* pa_status_string(int status);

/*
 * Read the current device's error word: *code gets a PA_DEVERR_* value,
 * *detail the offending index (token, request or block position). With
 * clear != 0 the word is reset. Synchronises the device; not for the hot path.
 * Either output pointer may be NULL.
 * There is one error word per device, in the library's static device memory,
 * shared by every call on that device whatever its stream: the first error
 * recorded since the last clear wins, so calls running concurrently on
 * different streams cannot tell whose error it is, and a clear resets it for
 * all of them. (The word's address is cached at the first call on a device;
 * the library does not support cudaDeviceReset of a device it has used.)
 */
pa_status pa_get_device_error(int* code, long long* detail, int clear);

/*
 * Device address of pinned host memory (cudaHostAlloc / cudaHostRegister,
 * mapped into the device's address space): the address kernels use to reach
 * it, which `out` of the attention calls accepts. PA_ERR_INVALID_ARG when
 * host_ptr is not pinned host memory or device_ptr is NULL; PA_ERR_CUDA on a
 * runtime error. *device_ptr is set only on success.
 */
pa_status pa_mapped_pointer(const void* host_ptr, void** device_ptr);

/*
 * Instrumentation: record `start_event` / `stop_event` (cudaEvent_t handles
 * created by the caller) around every later launch of the given kernel on its
 * stream; pass NULL events to stop. Kernel ids: 0 write_kv, 1 planner,
 * 2 decode (split-KV), 3 prefill chunk, 4 cascade prefix pass, 5 split-KV
 * merge pass, 6 accumulated weights, 7 eviction (these two: all launches of
 * the call), 8 reading back. Process-wide setting, not thread-safe.
 */
pa_status pa_set_kernel_timer(int kernel_id, void* start_event, void* stop_event);

/*
 * Process-wide options.
 *   PA_OPT_DECODE_SELF_PLAN (default 1): a batch whose spans are all at most
 *     one token (pure decode), with at most 512 requests and no cascade, is
 *     planned inside the split-KV kernel, and the planner is not launched.
 *     The results are bit-identical with the option off (the planner path),
 *     which the tests compare. value 0 turns it off.
 * PA_ERR_INVALID_ARG for an unknown option. Not thread-safe.
 */
#define PA_OPT_DECODE_SELF_PLAN 1
/*
 *   PA_OPT_DECODE_TC (default 1): which kernel runs the split-KV work (the
 *     decodes and the spans shorter than 16 tokens) at head_dim 128. 0: the
 *     CUDA-core kernel always. 1: the tensor-core kernel for GQA groups of 4
 *     or 8 query heads per KV head, over a bf16 or an E4M3 cache, where the
 *     CUDA cores' arithmetic per cached byte, not HBM, would set the pace;
 *     the CUDA-core kernel otherwise and for a cascade's suffix pass. 2: the
 *     tensor-core kernel wherever it applies (every group; cascade suffixes
 *     over a bf16 cache). Both give results within the attention tolerances
 *     of the exact result; they are not bit-identical to each other (the
 *     tensor-core kernel rounds P to bf16, or over an E4M3 cache splits the
 *     queries and 256 P into two E4M3 terms each, for its products).
 *   PA_OPT_DECODE_MAX_WORKERS (default 0, no cap): at most this many
 *     split-KV workers share the flattened (token, kv head, block) work, so
 *     a long sequence is split over fewer parts (1: none). For tests of the
 *     split-count invariance; the default uses every worker the launch has.
 *   PA_OPT_MIXED_OVERLAP (default 1): in a call with prefill chunks and
 *     split-KV work on the tensor-core split-KV kernel (bf16 cache), the
 *     planner may give the chunks a few SMs and the split-KV work the rest,
 *     so that both run at once (the mixed batch of "vLLM v1 Deep Dive",
 *     Part 3, Step 4c, whose prefill and decode spans one forward serves
 *     together). It does so when its cost
 *     model (per-SM prefill and split-KV rates measured on GB300) puts the
 *     two ending together sooner than one after the other, and otherwise runs
 *     them in turn as with the option off. The chunks' results are
 *     bit-identical either way; the split-KV results stay within the
 *     attention tolerances (fewer workers slice the keys differently).
 *     value 0 turns it off.
 */
#define PA_OPT_DECODE_TC 2
#define PA_OPT_DECODE_MAX_WORKERS 3
#define PA_OPT_MIXED_OVERLAP 4
/*
 *   PA_OPT_DECODE_TOKEN_MAJOR (default 1): over an E4M3 cache with eight KV
 *     heads at head_dim 128, the tensor-core split-KV kernel takes one 16-key
 *     block of all eight KV heads per tile (one tensor copy each for K and V,
 *     each head's keys in one half-warp). 0: the per-(token, kv head) tiles
 *     of the other groupings. Both are within the attention tolerances of
 *     the exact result on the same codes; they are not bit-identical.
 *     pa_attention_window_fp8 takes these tiles only for batches with enough
 *     decodes or keys attended to (G <= 4: a fifth as many decodes as SMs or 30
 *     blocks per SM; G = 8: three tenths, or 100 blocks per SM).
 */
#define PA_OPT_DECODE_TOKEN_MAJOR 5
/*
 *   PA_OPT_CASCADE_OVERLAP (default 1): in pa_attention_cascade, with the
 *     suffix pass on the CUDA-core split-KV kernel (the default routing), the
 *     prefix pass takes a few SMs (about two of its work items each) and the
 *     suffix pass the rest, both at once; every (token, kv head) then leaves
 *     fp32 partials and the merge pass folds suffix and prefix together.
 *     Results stay within the attention tolerances (the folding order
 *     differs). value 0: the prefix pass first, folded by the suffix pass.
 */
#define PA_OPT_CASCADE_OVERLAP 6
/*
 *   PA_OPT_DECODE_TM_CTAS_PER_SM (default 2; 1 or 2, anything else is
 *     PA_ERR_INVALID_ARG): CTAs per SM of the token-major E4M3 kernel. With 2
 *     (taken only at G = Hq / Hkv <= 4; G = 8 always runs one) each SM runs
 *     two CTAs of two copy stages each instead of one of four, so twice as
 *     many workers slice the keys; results stay within the attention
 *     tolerances. A windowed call below 64 blocks per SM runs one.
 */
#define PA_OPT_DECODE_TM_CTAS_PER_SM 7
/*
 *   PA_OPT_MIXED_PREFILL_CTAS (default 0; negative is PA_ERR_INVALID_ARG):
 *     in an overlapped mixed batch (PA_OPT_MIXED_OVERLAP), how many SMs the
 *     prefill chunks take beside the split-KV work. 0: the planner's cost
 *     model decides, and may run the two in turn instead. n > 0: always
 *     overlap, with min(n, SMs / 2) SMs for the chunks. Results do not depend
 *     on it beyond the attention tolerances (the split-KV slicing changes).
 */
#define PA_OPT_MIXED_PREFILL_CTAS 8
/*
 *   PA_OPT_WRITE_OVERLAP (default 0; 0 or 1, anything else is
 *     PA_ERR_INVALID_ARG): 1 lets the attention calls start beside the grid
 *     before them on the stream. A self-planned decode then streams K/V at once
 *     and waits for that grid only before a request's last block, where the
 *     newest token lies; a planner, a cascade's prefix pass and the splitting
 *     of the queries over an E4M3 cache start at once too. The caller promises
 *     that the work enqueued right before every attention call writes nothing
 *     that the call reads but the new tokens' K and V rows (and scales):
 *     pa_write_kv[_fp8, _rows] is such work, pa_norm_rope_write_kv (it makes q), pa_evict_kv and a
 *     kernel that makes q, lengths or tables are not. With 0 every call reads
 *     what the stream's work before it has written, whatever that is. Results
 *     are bit-identical. Llama-8B decode step: 99.6 us with 0, 98.0 with 1;
 *     over an E4M3 cache 68.8 and 64.8.
 */
#define PA_OPT_WRITE_OVERLAP 9
/*
 *   PA_OPT_SHARED_MIN_KB (default 24576; negative is PA_ERR_INVALID_ARG): a
 *     pa_attention_shared call whose groups would save less reading of K and V
 *     than this many KB - for every round of its work that the SMs take, where
 *     there are many groups - and hold no shared prefix of 4096 keys or more, attends
 *     without sharing: the prefix pass would cost more than it saves. 0: every
 *     group of two tokens shares. Results stay within the attention tolerances.
 */
#define PA_OPT_SHARED_MIN_KB 10
pa_status pa_set_option(int option, int value);

/* Number of kernel launches the library has issued in this process. */
long long pa_launch_count(void);

/* Library ABI version (major * 10000 + minor * 100 + patch). */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_API_H */
