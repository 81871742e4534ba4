/*
 * pa_int8_cache.h - a paged cache of 8-bit integers with a scale for every token
 * and KV head: written, read back, and attended over (C ABI).
 *
 * The pages list quantisation among vLLM's features without a format; this is
 * the library's second reading of it.  Against the E4M3 pools of pagedattn.h, whose
 * one scale per pool must be known beforehand, every row (one token, one KV
 * head, K or V) brings its own, taken as it is written.
 *
 *   scale = max_d |x[d]| / 127 (float32)     code[d] = x[d] / scale, to the nearest
 *   integer, ties to even, decided as in exact arithmetic     value = code * scale
 *
 * A row of zeros has scale 0.  A row that holds an infinity or NaN has scale
 * NaN and codes 0: all of it reads as NaN.  (A row with the largest float32 itself
 * has a scale that was rounded up: code 127 reads as an infinity there.)
 *
 * k_cache, v_cache    int8 [num_physical_blocks, block_size, num_kv_heads, head_size]
 * k_scales, v_scales  float [num_physical_blocks, num_kv_heads, block_size]: a
 *                     block's scales of one head side by side.  Attention wants them
 *                     16-byte aligned (PA_ERR_INVALID_ARG), writing and reading back
 *                     4-byte: allocate them 16-byte aligned.
 *
 * Copy-on-write of a forked sequence's block (pa_bm_append): pa_copy_blocks copies
 * bits, so the pools go through it as PA_BF16 with half the head_size, the scales as
 * PA_F32 with head_size 1 (block_size * num_kv_heads a multiple of 4 there).
 *
 * Conventions are those of pagedattn.h and pa_prefill.h.
 */
#ifndef PA_INT8_CACHE_H
#define PA_INT8_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "pa_prefill.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pa_write_cache_int8 - pa_write_cache into the int8 pools: row i of k_new and
 * v_new goes to slot_mapping[i] as codes and scales.
 * k_new, v_new  [num_tokens, num_kv_heads, head_size], PA_BF16 or PA_F32 (src_dtype),
 *               16-byte aligned
 * slot_mapping  [num_tokens] int64; negative: padding; beyond the pool: skipped
 *               and reported (PA_DEVERR_SLOT).  Of two rows with one slot either
 *               may remain, codes and scales possibly not of the same one.
 * head_size 64 or 128; pools 16-byte, scales 4-byte aligned.
 */
int pa_write_cache_int8(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                        void* k_cache, void* v_cache, float* k_scales, float* v_scales, int num_tokens,
                        int num_kv_heads, int head_size, int block_size, int num_physical_blocks,
                        void* stream, int src_dtype, int32_t* error_flag);

/*
 * pa_read_cache_int8 - tokens of the sequences, read back through their block
 * tables into plain rows: row seq_starts[s] + i of k_out and v_out becomes token
 * first_tokens[s] + i of sequence s, for i < seq_starts[s + 1] - seq_starts[s].
 * k_out, v_out  [num_tokens, num_kv_heads, head_size], PA_BF16 or PA_F32 (dst_dtype);
 *               code * scale in float32, rounded once to bf16.  Rows before the
 *               first and behind the last sequence's are left as they are.
 * first_tokens  [num_seqs] int32, or NULL: 0
 * seq_starts    [num_seqs + 1] int32, as in pa_prefill; where entries decrease, a row
 *               may be left as it is (PA_DEVERR_CONTEXT_LEN)
 * A token outside its sequence's row of the tables (PA_DEVERR_CONTEXT_LEN), or of a
 * block outside the pool (PA_DEVERR_BLOCK_ID; num_physical_blocks > 0 is
 * required), leaves its row as it is.
 * The rows, which are a pool of num_tokens blocks of one token, are what attention
 * of the framework's other pool types can run over.
 */
int pa_read_cache_int8(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                       const float* k_scales, const float* v_scales, const int32_t* block_tables,
                       const int32_t* first_tokens, const int32_t* seq_starts, int num_tokens,
                       int num_seqs, int num_kv_heads, int head_size, int block_size,
                       int max_blocks_per_seq, int num_physical_blocks, void* stream, int dst_dtype,
                       int32_t* error_flag);

/*
 * pa_prefill_int8 - pa_prefill over the int8 pools; query and out bf16.  Codes
 * enter both products exactly (as bf16 integers), K's scales multiply the scores
 * and V's the weights in fp32, and the products weight * scale are rounded to bf16
 * (at most 2^-8 of themselves, as long as V's scale is above 2^-110: a weight may
 * enter as 2^-16 of itself, and bf16 ends at 2^-126; rows that pa_prefill carries in two parts: 2^-16).  A token whose scale is NaN makes the rows that see it NaN, and
 * no others.  num_physical_blocks > 0 is required.  Other arguments, scratch
 * and limits as in pa_prefill.
 *
 * pa_decode_int8 - one decode step over the int8 pools: num_queries new tokens for every
 * sequence, query and out [num_seqs, num_queries, num_heads, head_size], results as
 * of pa_prefill_int8.  As in pa_decode_fp8_mq the query is rounded to f16 (exact
 * for |q| in [2^-14, 65504]) and so are the softmax weights times V's scales: off by
 * at most 2^-11 of themselves or 2^-38 of the largest weight times the largest scale,
 * whichever is more.  A row is finite as long as the sum of its weights (the largest counted as
 * 1) times |v| is, whatever the values.  More than 32
 * (query, head) columns per KV head, or head_size 64 with an odd num_kv_heads, run as
 * chunks do (pa_prefill_int8).
 * workspace    as in pa_decode_ws: at least pa_decode_int8_workspace_size(...) bytes,
 *              zero-filled before its first use and reusable as it is behind every call,
 *              by other shapes, too; or NULL: the library's own, one buffer per stream, as in
 *              pa_prefill (refused while `stream` is being captured)
 * num_ranges   as in pa_decode_ex (shapes that run as chunks: without effect)
 */
int pa_prefill_int8(void* out, const void* query, const void* k_cache, const void* v_cache,
                    const float* k_scales, const float* v_scales, const int32_t* block_tables,
                    const int32_t* context_lens, const int32_t* seq_starts, int num_tokens, int num_seqs,
                    int num_heads, int num_kv_heads, int head_size, int block_size,
                    int max_blocks_per_seq, float scale, void* stream, int num_physical_blocks,
                    void* workspace, size_t workspace_bytes, int32_t* error_flag);
int pa_decode_int8(void* out, const void* query, const void* k_cache, const void* v_cache,
                   const float* k_scales, const float* v_scales, const int32_t* block_tables,
                   const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                   int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq, float scale,
                   void* stream, int num_physical_blocks, void* workspace, size_t workspace_bytes,
                   int num_ranges, int32_t* error_flag);

/* Scratch bytes pa_decode_int8 needs on the current device (0 for invalid sizes). */
size_t pa_decode_int8_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                     int head_size, int num_ranges);

#ifdef __cplusplus
}
#endif

#endif /* PA_INT8_CACHE_H */
