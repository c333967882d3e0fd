/*
 * fp8amax_serving.h - C ABI of what a serving step runs between the FP8 projections: the
 * bookkeeping of a paged key/value cache, the rotation of queries and keys by their positions,
 * the write of new keys and values into the cache, and causal attention over whole prompts or
 * over the cache, for MI355X (gfx950).  Same library,
 * status codes and conventions as fp8amax.h: device pointers owned by the caller, nothing
 * allocated and no state kept, arguments validated on the host before any HIP call, all work
 * enqueued on `stream`, no synchronisation, capturable in a HIP graph.
 *
 * The cache.  K and V each hold `pages` pages of `page_size` tokens,
 *   cache[page][kv_head][token in page][head_dim],
 * in one of three formats:
 *   FP8_KV_SAME: the 16-bit type of the new keys and values;
 *   FP8_KV_E4M3: uint8 e4m3fn codes and one float32 scale per token and head,
 *     scales[page][kv_head][token in page]; value = code * scale, with scale and codes by the
 *     rules of fp8amax.h over the head_dim values (scale = amax / 448, 1 for an all-zero row);
 *   FP8_KV_MXFP4: e2m1 codes, two a byte (an even channel in the low half), in rows of head_dim / 2
 *     bytes, and one scale byte s for a token, head and 32 channels, scales[page][kv_head][token in
 *     page][head_dim / 32]; value = {0, 0.5, 1, 1.5, 2, 3, 4, 6}[code & 7] * 2^(s - 127), negative with
 *     bit 3 of the code, and NaN with s = 255.  As written: 2^(s - 127) is the smallest power of two
 *     (from 2^-127) not below a block's amax / 6, 1 (s = 127) for an all-zero block, and each code the
 *     one nearest to x / 2^(s - 127), ties to the even code; where 4 times the scale is past dt's
 *     range (a block's amax from 3 / 4 of 2^16 in fp16, of 2^128 in bf16) no larger than 3.  A block that
 *     holds a value that is not finite has s = 255 and codes 0.
 * A token's slot is page * page_size + (token in page).  Request r's tokens p, p + 1, .. lie in
 * the pages block_table[r][p / page_size] (row-major [batch, width]); entries that name no
 * page of the cache are allowed: what they hold reads as zero and is never written.
 *   page_size : a power of two, 16 .. 1024.
 *   head_dim  : 64 or 128.
 *   q_heads   : a multiple of kv_heads; query head h reads key head h / (q_heads / kv_heads).
 *   dt        : bf16 or fp16, the type of q, k, v and the output.
 *
 * Packed sequences.  The tokens of a step's requests lie one after the other; request r's are
 * [cu_tokens[r], cu_tokens[r + 1]) (int32 [batch + 1] on the device, non-decreasing from 0).
 * Values outside [0, tokens] are clamped and a request whose end precedes its start is empty,
 * so any values give in-bounds accesses; what is computed where they decrease is not specified.
 * Output rows that no request covers are not written.
 *
 * Strides.  q, k and v are [tokens, heads, head_dim] with the last index contiguous; the token
 * and head strides are given in elements, non-negative multiples of 8 (so that a fused
 * projection's output is read in place).  Data pointers need 16-byte, int32, float32
 * and scale pointers 4-byte, int64 pointers 8-byte alignment.
 *
 * What a call writes shares no memory with what it reads or else writes; an append refuses caches and
 * scales that share memory with each other (FP8_ERR_BAD_SHAPE), but for fp8_kv_append of one tensor as k
 * and v into one cache.
 *
 * Sizes.  FP8_ERR_TOO_LARGE, before any HIP call, where tokens * heads passes 2^30 or the work would
 * need 2^24 workgroups or more (a launch holds less than 2^32 threads): a workgroup appends 16 rows
 * of 128 channels or 32 of 64 (with rotation at least as many), and attends for 128 rows or 32 of one request and key
 * head (16 over FP8_KV_MXFP4).
 */
#ifndef FP8AMAX_SERVING_H
#define FP8AMAX_SERVING_H

#include "fp8amax.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum FP8_ENUM_BASE { FP8_KV_SAME = 0, FP8_KV_E4M3 = 1, FP8_KV_MXFP4 = 4 } fp8_kv_format_t;

/*
 * fp8_paged_plan - block tables, slots and positions of one step, in one launch, from the
 * requests' lengths on the device.
 *   cached, added : int32 [batch], a request's tokens in the cache before the step and its new
 *                 tokens; negative values count as 0.
 *   block_table : int32 [batch, width], in and out: the pages of the cached tokens are read,
 *                 and the entries ceil(cached / page_size) .. ceil((cached + added) / page_size)
 *                 get pages from the free list, in the order of the requests; others stay.
 *   free_pages  : int32 [n_free]; taken_in int32 [1]: how many of them are in use already.
 *   taken_out   : int32 [1], taken_in plus the pages given out.
 *   missing     : int32 [1], pages that were needed and not given: the free list was used up
 *                 (their entries become -1) or the table has no entry for them.
 *   cu_tokens   : int32 [batch + 1], the prefix sums of `added`.
 *   seq_lens    : int32 [batch], cached + added.
 *   positions   : int32 [tokens], each new token's position in its request, -1 past the last.
 *   slots       : int64 [tokens], each new token's slot; -1 past the last token and for tokens
 *                 without a page.
 * The outputs, block_table among them, share no memory with an input or with each other (refused as
 * FP8_ERR_BAD_SHAPE): lengths are not advanced in place, nor is taken_in.
 * tokens is the size of positions and slots; new tokens past it are counted in cu_tokens only.
 * batch <= 16384; batch == 0 fills positions and slots with -1.  Requires width >= 1.
 */
fp8_status_t fp8_paged_plan(const int32_t* cached, const int32_t* added, int64_t batch, int32_t page_size,
                            int32_t* block_table, int64_t width, const int32_t* free_pages, int64_t n_free,
                            const int32_t* taken_in, int64_t tokens, int32_t* cu_tokens, int32_t* seq_lens,
                            int32_t* positions, int64_t* slots, int32_t* taken_out, int32_t* missing, void* stream);

/*
 * fp8_kv_append - new keys and values into the pages of their slots, as they are or quantized,
 * in one launch.
 *   k, v    : [tokens, kv_heads, head_dim] of dt, strided.
 *   slots   : int64 [tokens]; a slot outside [0, pages * page_size) is skipped (-1: padding).
 *             Two tokens with one slot leave parts of either's row there (a scale and codes that are not
 *             of one token, too): a step's slots differ.
 *   k_cache, v_cache : as above; k_scales, v_scales : float32 (FP8_KV_E4M3) or bytes (FP8_KV_MXFP4),
 *   NULL for FP8_KV_SAME.
 */
fp8_status_t fp8_kv_append(const void* k, const void* v, fp8_dtype_t dt, int64_t tokens, int64_t kv_heads,
                           int32_t head_dim, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                           int64_t v_head_stride, const int64_t* slots, int64_t pages, int32_t page_size,
                           fp8_kv_format_t format, void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                           void* stream);

/*
 * fp8_rope_append - fp8_kv_append with the position rotation on the way: the queries and keys of a
 * step rotated by their positions, the queries into q_out, the keys with their values into the
 * pages of their slots, in one launch.  With R = rotary_dim and row p of the table,
 *   cos_sin[p] = cos_0 .. cos_(R/2 - 1), sin_0 .. sin_(R/2 - 1),
 * a token at position p gets, for i < R / 2,
 *   x'_a = x_a cos_i - x_b sin_i,   x'_b = x_b cos_i + x_a sin_i,
 *   (a, b) = (i, i + R / 2), or (2 i, 2 i + 1) with interleaved != 0;
 * channels from R on stay.  Products and sums are float32 (each rounded once); q_out and a cache of
 * FP8_KV_SAME get the result rounded once to dt, the other formats quantize the float32 result.
 *   q       : [tokens, q_heads, head_dim] of dt, strided; q_heads may be 0 (q and q_out unused) and
 *             need not be a multiple of kv_heads.
 *   q_out   : [tokens, q_heads, head_dim] of dt, dense.
 *   positions : int32 [tokens]; a token whose position is outside [0, n_positions) is skipped: neither
 *             q_out nor the cache is written.  One with a position but without a slot (as in
 *             fp8_kv_append) gets its queries.
 *   cos_sin : float32 [n_positions, R], 16-byte aligned; R a multiple of 16, 16 .. head_dim.
 * Other arguments as fp8_kv_append.
 */
fp8_status_t fp8_rope_append(const void* q, const void* k, const void* v, fp8_dtype_t dt, int64_t tokens,
                             int64_t q_heads, int64_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                             int64_t q_head_stride, int64_t k_token_stride, int64_t k_head_stride,
                             int64_t v_token_stride, int64_t v_head_stride, const int32_t* positions,
                             const float* cos_sin, int64_t n_positions, int32_t rotary_dim, int32_t interleaved,
                             const int64_t* slots, int64_t pages, int32_t page_size, fp8_kv_format_t format,
                             void* k_cache, void* v_cache, void* k_scales, void* v_scales, void* q_out,
                             void* stream);

/*
 * fp8_attn_prompt - causal attention over whole prompts.  For query i of a request, over the
 * keys j <= i of the same request (with window > 0: i - window < j <= i):
 *   out_i = sum_j softmax_j(softmax_scale * q_i . k_j) v_j
 *   lse_i = log sum_j exp(softmax_scale * q_i . k_j)
 *   out : [tokens, q_heads, head_dim] of dt, dense.  lse : NULL or float32 [tokens, q_heads].
 *   The token strides of k and v are at least head_dim (with more than one token) and at most 2^20.
 *   softmax_scale : finite and > 0.
 *   window : 0 (none; 2^30 or more is none too) or the number of keys a query sees at most.
 * Scores, the running maximum and sum, and the output accumulate in float32; the weights are
 * rounded to dt for the product with v, and the result once to dt.  Over a cache in FP8_KV_E4M3 a
 * key's scale multiplies its score in float32, and a value's scale its weight before that rounding;
 * with fp16 the scale's power of two, from 2^-14 to 2^7, multiplies the codes instead, exactly.
 * Over FP8_KV_MXFP4 keys and values enter as numbers of dt: exactly with bf16, and with fp16 for
 * scales from 2^-23 to 2^13 (below, rounded to its subnormal numbers; values past its range are
 * infinite).
 */
fp8_status_t fp8_attn_prompt(const void* q, const void* k, const void* v, fp8_dtype_t dt, int64_t tokens,
                             const int32_t* cu_tokens, int64_t batch, int64_t q_heads, int64_t kv_heads,
                             int32_t head_dim, int64_t q_token_stride, int64_t q_head_stride,
                             int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                             int64_t v_head_stride, float softmax_scale, int64_t window, void* out, float* lse,
                             void* stream);

/*
 * fp8_attn_paged - the same for each request's new tokens over its pages: the n new tokens of
 * a request of seq_lens[r] tokens in the cache (the new ones among them) are its last n, so
 * query i of them sits at position seq_lens[r] - n + i and sees the keys up to there.  A query
 * at a negative position (seq_lens[r] < n) sees none: its output is 0 and its lse -inf.
 *   seq_lens : int32 [batch], clamped to [0, width * page_size], which is at most 2^30.
 *   max_new  : the largest number of new tokens of a request, 0 if unknown; it chooses the
 *              kernel and has no effect on what is computed.
 *   workspace : workspace_bytes of device memory, 16-byte aligned, of at least
 *              fp8_attn_paged_workspace() bytes for the same sizes (may be 0).  Its first
 *              FP8_ATTN_COUNTER_BYTES must be zero before the first call; every call leaves it fit
 *              for the next one, of the same or of other sizes.  Calls that may run at the same time
 *              need different ones.
 */
#define FP8_ATTN_COUNTER_BYTES 16384

int64_t fp8_attn_paged_workspace(int64_t tokens, int64_t batch, int64_t q_heads, int64_t kv_heads, int32_t head_dim,
                                 int64_t width, int32_t page_size, int64_t max_new);

fp8_status_t fp8_attn_paged(const void* q, fp8_dtype_t dt, int64_t tokens, const int32_t* cu_tokens, int64_t batch,
                            int64_t q_heads, int64_t kv_heads, int32_t head_dim, int64_t q_token_stride,
                            int64_t q_head_stride, fp8_kv_format_t format, const void* k_cache, const void* v_cache,
                            const void* k_scales, const void* v_scales, int64_t pages, int32_t page_size,
                            const int32_t* block_table, int64_t width, const int32_t* seq_lens, float softmax_scale,
                            int64_t window, int64_t max_new, void* out, float* lse, void* workspace,
                            int64_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* FP8AMAX_SERVING_H */
