/*
 * gqa_cache.h - what happens to a KV cache's rows around the attention of
 * gqa.h: the norm and rotation of query and key heads on the way in, the
 * attention weight each row collects, the eviction of the rows that collect
 * least, and a cache of microscaled 4-bit values. Same library (libgqa.so),
 * same notation and conventions as gqa.h: device pointers, 16-byte aligned
 * contiguous tensors unless a stride is given, caller-owned buffers and
 * workspaces, asynchronous on `stream`, device-side problems reported through
 * gqa_get_last_error(). All calls may be captured into a CUDA graph.
 *
 * Workspaces need no initialisation and carry nothing from one call to the
 * next. A size that a gqa_*_workspace_bytes call here returns for a batch of B
 * also serves every smaller batch of the same other arguments. Two calls (or replays of graphs) that share a workspace must not
 * overlap on the GPU.
 */
#ifndef GQA_CACHE_H_
#define GQA_CACHE_H_

#include "gqa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* One more bit of the device error word. */
#define GQA_DEVERR_ROPE_POS 0x10u /* gqa_qk_norm_rope: a position outside [0, max_pos); the nearest table row was used */

/*
 * gqa_rope_table - the table of a position rotation.
 *
 *   rope[p, i]                  = cos(p * theta^(-2 i / rotary_dim))
 *   rope[p, rotary_dim / 2 + i] = sin(p * theta^(-2 i / rotary_dim)),  i < rotary_dim / 2
 *
 * Angles, cosines and sines are computed in 64 bits and rounded once, so far
 * positions lose nothing. Callers with scaled frequencies fill the table
 * themselves; gqa_qk_norm_rope reads only its values.
 *
 * rope : [max_pos, rotary_dim] float32, written. rotary_dim is even, > 0.
 */
GQA_API int gqa_rope_table(float* rope, int max_pos, int rotary_dim, double theta, gqa_stream_t stream);

/*
 * gqa_qk_norm_rope - the norm of every query and key head, the position
 * rotation, and the new rows' way into the cache, in one pass.
 *
 *   y = x / sqrt(mean_i x_i^2 + eps) * w      (skipped where the weight is NULL)
 *   (y_i, y_j) -> (y_i cos_i - y_j sin_i, y_j cos_i + y_i sin_i),  i < rotary_dim / 2
 *   with j = i + rotary_dim / 2, or for interleaved != 0 the pair (2 i, 2 i + 1);
 *   dims from rotary_dim on are not rotated.
 *
 * float32 arithmetic (a row's squares and their sum have to lie in its range),
 * one rounding to dtype at the end.
 *
 * q, k, v    : T new tokens of each of B sequences; token n = b * T + t
 *              starts q_stride (k_stride, v_stride) elements after token
 *              n - 1, its H (K) heads of d elements contiguous: slices of
 *              one fused projection's output will do. Strides are multiples
 *              of 16 bytes and at least one token's heads.
 * q_out      : [B, T, H, d], written. May be q itself (q_stride = H * d).
 * k_out      : [B, T, K, d] or NULL: the keys for a prefill. May be k itself.
 * k_cache,
 * v_cache    : [B, K, S_max, d] or both NULL. When given, token t of sequence
 *              b goes to row rows[b] + t: its finished keys, and v as it is.
 * row_pos    : [B, K, S_max] int32 or NULL: row rows[b] + t is set to the
 *              token's position (what gqa_kv_evict knows a row's age by).
 * q_weight,
 * k_weight   : [d] of dtype, or NULL (no norm).
 * rope       : [max_pos, rotary_dim] float32 (gqa_rope_table). rotary_dim is
 *              a multiple of 16, at most d; 0 means no rotation (rope may
 *              then be NULL).
 * positions  : [B, T] int32, device. One outside [0, max_pos) sets
 *              GQA_DEVERR_ROPE_POS and uses the nearest table row. Not read
 *              when rotary_dim is 0 and row_pos is NULL.
 * rows       : [B] int32, device; needed with a cache or row_pos. Where
 *              rows[b] < 0 or rows[b] + T > S_max, GQA_DEVERR_APPEND_POS is
 *              set and sequence b's cache rows and row_pos are left as they
 *              are (q_out and k_out are written). A cache that gqa_kv_evict
 *              has cut has rows below their positions.
 * The paged form writes into a pool and its table (gqa.h, paged KV cache);
 * row_pos there is [B, K, max_blocks * block_size], by logical row. A table
 * entry outside the pool sets GQA_DEVERR_BLOCK and drops the row.
 */
GQA_API int gqa_qk_norm_rope(void* q_out, void* k_out, void* k_cache, void* v_cache, int32_t* row_pos, const void* q,
                             const void* k, const void* v, const void* q_weight, const void* k_weight,
                             const float* rope, const int32_t* positions, const int32_t* rows, int B, int T, int H,
                             int K, int S_max, int d, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             int rotary_dim, int max_pos, int interleaved, float eps, gqa_dtype dtype,
                             gqa_stream_t stream);
GQA_API int gqa_qk_norm_rope_paged(void* q_out, void* k_out, void* k_pool, void* v_pool, int32_t* row_pos,
                                   const void* q, const void* k, const void* v, const void* q_weight,
                                   const void* k_weight, const float* rope, const int32_t* positions,
                                   const int32_t* block_table, const int32_t* rows, int B, int T, int H, int K,
                                   int d, int num_blocks, int block_size, int max_blocks, int64_t q_stride,
                                   int64_t k_stride, int64_t v_stride, int rotary_dim, int max_pos, int interleaved,
                                   float eps, gqa_dtype dtype, gqa_stream_t stream);

/*
 * gqa_decode_scores - gqa_decode, and what each cached row got of the
 * attention added to its score:
 *
 *   p[b,h,t]      = softmax_{t < len_b}(scale * q[b,h,:] . k[b,g,t,:])
 *   out[b,h,:]    = sum_t p[b,h,t] v[b,g,t,:]
 *   scores[b,g,t] += sum_{h in group g} p[b,h,t],   t < len_b
 *
 * scores : [B, K, S_max] float32, in place. Scores of rows t >= len_b are
 *          neither read nor written; a row that joins the cache starts from
 *          what the caller (or gqa_kv_evict) left there, normally 0. The sum
 *          over a group's heads is taken in a fixed order: results repeat
 *          bit for bit.
 * Sums are float32; a weight meets the values rounded by 2^-15 of itself.
 * A key whose score is -inf weighs nothing. A query head that has no other
 * key adds nothing to the scores and its output is zeros, as for an empty
 * sequence. A NaN score makes all of its head's weights and its output NaN.
 * The paged form's scores are [B, K, max_blocks * block_size], by logical
 * row. Everything else as for gqa_decode and gqa_decode_paged; GQA_BF16 only
 * (GQA_F32 returns GQA_ERR_UNSUPPORTED).
 * workspace : gqa_decode_scores_workspace_bytes(...) bytes: the partial
 *          results and one float per query head and row of the cache. 0 for
 *          invalid shapes.
 */
GQA_API size_t gqa_decode_scores_workspace_bytes(int B, int H, int K, int S_max, int d, int num_splits);
GQA_API int gqa_decode_scores(void* out, float* scores, const void* q, const void* k_cache, const void* v_cache,
                              const int32_t* seqlens, int B, int H, int K, int S_max, int d, float scale,
                              int num_splits, void* workspace, size_t workspace_bytes, gqa_dtype dtype,
                              gqa_stream_t stream);
GQA_API size_t gqa_decode_scores_paged_workspace_bytes(int B, int H, int K, int d, int block_size, int max_blocks,
                                                       int num_splits);
GQA_API int gqa_decode_scores_paged(void* out, float* scores, const void* q, const void* k_pool, const void* v_pool,
                                    const int32_t* block_table, const int32_t* seqlens, int B, int H, int K, int d,
                                    int num_blocks, int block_size, int max_blocks, float scale, int num_splits,
                                    void* workspace, size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream);

/*
 * gqa_prompt_scores - the scores that the last T tokens of each sequence add
 * (T = the prompt's length: the whole prompt; a small T: an observation
 * window), without their attention output:
 *
 *   scores[b,g,t] += sum_{i < T} sum_{h in group g} p[b,i,h,t]
 *   p[b,i,h,:]     = softmax over t <= len_b - T + i of scale * q[b,i,h,:] . k[b,g,t,:]
 *
 * q       : [B, T, H, d]; query i of sequence b is its token len_b - T + i.
 *           Where that is negative (a prompt shorter than T, its queries at
 *           the end of the T) the query does not count and is not read into
 *           the result.
 * k_cache : [B, K, S_max, d], row t the key of token t (no row evicted yet).
 * seqlens : [B] int32, device; outside [0, S_max] sets GQA_DEVERR_SEQLEN and
 *           leaves the sequence's scores as they are.
 * scores  : [B, K, S_max] float32, in place; rows t >= len_b are neither
 *           read nor written. Results repeat bit for bit.
 * Keys at -inf and NaN as in gqa_decode_scores: a query that sees keys at -inf
 * alone (the padding of a left-padded prompt, masked by its keys) adds nothing.
 * GQA_BF16 only, H / K at most 128 (GQA_ERR_SHAPE). workspace:
 * gqa_prompt_scores_workspace_bytes(...) bytes.
 */
GQA_API size_t gqa_prompt_scores_workspace_bytes(int B, int T, int H, int K, int S_max, int d);
GQA_API int gqa_prompt_scores(float* scores, const void* q, const void* k_cache, const int32_t* seqlens, int B, int T,
                              int H, int K, int S_max, int d, float scale, void* workspace, size_t workspace_bytes,
                              gqa_dtype dtype, gqa_stream_t stream);

/*
 * gqa_kv_evict - cut each sequence of more than `keep` rows to `keep` rows,
 * every KV head on its own: the rows that collected least go.
 *
 * Rows t < len_b of (b, g) are ranked: first the held rows (position < sinks,
 * or position >= recent_from[b]), the lower row first; then the others by
 * score, the higher first, the lower row first among equal scores (-0 equals
 * 0; a NaN counts below every number). The first `keep` stay. Of those, the
 * ones in rows >= keep move, in order of their rows, into the rows below keep
 * that were given up, in order; the others stay where they are: only as many
 * rows move as have to, and the order of the rows is not kept (a decode over
 * the cache does not depend on it, and row_pos says which is which).
 *
 * k_cache, v_cache : [B, K, S_max, d] of dtype, in place. Rows >= keep are
 *                    left as they are.
 * scores      : [B, K, S_max] float32, moved along; rows keep <= t < len_b of
 *               a cut sequence become 0, ready for new tokens.
 * row_pos     : [B, K, S_max] int32 or NULL, the position of each row's
 *               token, moved along; rows keep <= t < len_b become -1. NULL: a
 *               row's position is its index (a cache cut for the first time).
 * seqlens     : [B] int32, device, in place: min(len_b, keep) afterwards. A
 *               value outside [0, S_max] sets GQA_DEVERR_SEQLEN and the
 *               sequence is left as it is.
 * recent_from : [B] int32, device, or NULL (no row is held for its age).
 * keep        : 1 <= keep <= S_max. sinks : >= 0.
 * workspace   : gqa_kv_evict_workspace_bytes(...) bytes (S_max =
 *               max_blocks * block_size for the paged form); 0 if invalid.
 * The paged form moves rows between the blocks of the table; the blocks must
 * not be shared with another sequence. A table entry outside the pool sets
 * GQA_DEVERR_BLOCK and the move of its row is dropped.
 */
GQA_API size_t gqa_kv_evict_workspace_bytes(int B, int K, int S_max, int keep);
GQA_API int gqa_kv_evict(void* k_cache, void* v_cache, float* scores, int32_t* row_pos, int32_t* seqlens,
                         const int32_t* recent_from, int B, int K, int S_max, int d, int keep, int sinks,
                         void* workspace, size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream);
GQA_API int gqa_kv_evict_paged(void* k_pool, void* v_pool, const int32_t* block_table, float* scores, int32_t* row_pos,
                               int32_t* seqlens, const int32_t* recent_from, int B, int K, int d, int num_blocks,
                               int block_size, int max_blocks, int keep, int sinks, void* workspace,
                               size_t workspace_bytes, gqa_dtype dtype, gqa_stream_t stream);

/*
 * 4-bit KV cache: gqa_kv_append_mxfp4, gqa_kv_read_mxfp4, gqa_decode_mxfp4.
 *
 * Rows of microscaled 4-bit values (the MXFP4 format of the OCP Microscaling
 * Formats specification 1.0): blocks of 32 consecutive dims share a scale
 * 2^(E - 127), each value is an e2m1 code (sign, 0 0.5 1 1.5 2 3 4 6):
 *
 *   value[b, g, t, i] = e2m1(code i) * 2^(scales[b, g, t, i / 32] - 127)
 *
 * k_codes, v_codes   : [B, K, S_max, d / 2] uint8, code 2 j in the low half of
 *                      byte j, code 2 j + 1 in the high half.
 * k_scales, v_scales : [B, K, S_max, d / 32] uint8 exponents E (255: NaN).
 * d must be 128 (GQA_ERR_UNSUPPORTED) and S_max a multiple of 4
 * (GQA_ERR_SHAPE). A row is 68 bytes against 256 in bfloat16.
 *
 * gqa_kv_append_mxfp4 quantizes T new tokens' rows k_new, v_new ([B, T, K, d]
 * bfloat16) into rows pos[b] .. pos[b] + T - 1: 2^(E - 127) is the largest
 * power of two not above the block's largest magnitude, over 4 (E = 0 where
 * that lies below 2^-127); code = x / 2^(E - 127) rounded to nearest, ties to the
 * even code, magnitudes beyond 6 to 6, the sign kept. A block that holds a
 * NaN or an infinity gets E = 255 and codes 0: its values are NaN. pos[b] < 0
 * or pos[b] + T > S_max sets GQA_DEVERR_APPEND_POS and leaves that sequence's
 * rows unwritten.
 *
 * gqa_kv_read_mxfp4 reads rows pos[b] .. pos[b] + T - 1 back as bfloat16
 * ([B, T, K, d]; exact, but for codes of a foreign writer whose value passes
 * bfloat16's largest: infinity), for a prefill that goes on from a cached prompt. Out of range: GQA_DEVERR_APPEND_POS, zeros.
 *
 * gqa_decode_mxfp4 is gqa_decode over the values the 4-bit cache holds: q and
 * out are [B, H, d] bfloat16, everything else as for gqa_decode. Rows
 * t >= len_b are never read into the result. Sums are float32; a weight meets
 * the values with a rounding of at most 2^-9 of itself or 2^-28 of the largest
 * weight of its split. A key whose score falls below float32's range weighs
 * nothing; a head that has no other key gets zeros, as for an empty sequence.
 * (K block scales above 2^108 may take a score out of float32's range whatever
 * q is: a head's elements meet them at 2^8 times their share of its largest.)
 */
GQA_API int gqa_kv_append_mxfp4(uint8_t* k_codes, uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales,
                                const void* k_new, const void* v_new, const int32_t* pos, int B, int T, int K,
                                int S_max, int d, gqa_stream_t stream);
GQA_API int gqa_kv_read_mxfp4(void* k_out, void* v_out, const uint8_t* k_codes, const uint8_t* k_scales,
                              const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* pos, int B, int T, int K,
                              int S_max, int d, gqa_stream_t stream);
GQA_API size_t gqa_decode_mxfp4_workspace_bytes(int B, int H, int K, int S_max, int d, int num_splits);
GQA_API int gqa_decode_mxfp4(void* out, const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                             const uint8_t* v_codes, const uint8_t* v_scales, const int32_t* seqlens, int B, int H,
                             int K, int S_max, int d, float scale, int num_splits, void* workspace,
                             size_t workspace_bytes, gqa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GQA_CACHE_H_ */
