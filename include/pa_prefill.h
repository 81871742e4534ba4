/*
 * pa_prefill.h - attention of chunks of new tokens over the paged cache (C ABI).
 *
 * The step that "vLLM three-process architecture and the PagedAttention kernel"
 * (devpress.csdn.net) puts before decode (section 2: the prompt's tokens go
 * through the model first, a chunk per step where the token budget says so),
 * on the gather of its section 3.2.  A batch is ragged: every sequence brings
 * any number of new tokens, one (a decode), a prompt's chunk or none.
 *
 * Conventions are those of pagedattn.h: device pointers owned by the caller,
 * asynchronous on `stream`, PA_OK or a negative PA_ERR_* code with a message
 * in pa_last_error(), nothing queued on error.
 */
#ifndef PA_PREFILL_H
#define PA_PREFILL_H

#include <stddef.h>
#include <stdint.h>

#include "pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pa_prefill - causal attention of every sequence's newest tokens over its
 * paged keys and values.
 *
 * Sequence s has n = seq_starts[s + 1] - seq_starts[s] new tokens; its token i is
 * row seq_starts[s] + i of query and out, and sits at position
 * context_lens[s] - n + i:
 *
 *   out[row, h, :] = sum_t softmax_t(scale * <query[row, h, :], K_s[t, h/G, :]>) V_s[t, h/G, :]
 *                    over t = 0 .. context_lens[s] - n + i
 *
 * out, query   [num_tokens, num_heads, head_size], dtype
 * seq_starts   [num_seqs + 1] int32, not decreasing, within 0 .. num_tokens, as
 *              pa_tables_step writes them.  Rows before the first and behind the
 *              last are neither read nor written.
 * context_lens [num_seqs] int32: every valid token, the new ones included, whose
 *              K/V must be in the pool already (pa_write_cache)
 * Other tensors as in pa_decode.  A row whose position is negative (a context
 * shorter than its new tokens) becomes zero.  A sequence whose entries of
 * seq_starts decrease or leave 0 .. num_tokens gets the rows that remain of them
 * and is reported (PA_DEVERR_CONTEXT_LEN), as lengths outside the tables are.
 * A token that some new token of its sequence sees must be finite for the
 * others too (its weight there is zero, but zero times NaN is NaN).
 * Types: PA_BF16 or PA_F32.  num_heads / num_kv_heads <= 8, head_size 64 or 128,
 * block_size 1 .. 4096 (multiples of 8 stream fastest), num_tokens *
 * num_heads < 2^31.  bf16: the softmax weights enter the second product rounded to
 * bf16 (at most 2^-8 of themselves), the sums keep them in fp32.  A chunk's tokens go
 * in tiles of t = 128 / (num_heads / num_kv_heads), two at a time; a tile that is left
 * alone (all of a chunk of at most t tokens, a decode for one) carries the weights in two
 * bf16 parts, 2^-16 together.  So a token's rounding depends on the chunk that it comes in.
 * Weights under 2^-110 of a row's largest (fp32 pools: 2^-126) may count as zero.  A row
 * is finite as long as the sum of its weights (the largest counted as 1) times |v| is.
 * num_physical_blocks > 0: block ids are checked against it, and tokens of a
 * bad one are unspecified; 0: as in pa_decode_ex.
 * workspace    256-byte aligned device scratch of at least
 *              pa_prefill_workspace_size(...) bytes, of any content (the first
 *              16 KiB are left alone: see pa_decode_ws); two calls that may
 *              overlap in time must not share it.  NULL: the library's
 *              own, one buffer per stream, as in pa_decode_mod (refused while
 *              `stream` is being captured).
 * The call makes two launches: the attention, whose list of (row tile, token
 * tile) pairs is cut into equal ranges, one per SM, and the join of the rows
 * that such a cut divides.
 */
int pa_prefill(void* out, const void* query, const void* k_cache, const void* v_cache,
               const int32_t* block_tables, const int32_t* context_lens, const int32_t* seq_starts,
               int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_size,
               int block_size, int max_blocks_per_seq, float scale, void* stream, int dtype,
               int num_physical_blocks, void* workspace, size_t workspace_bytes, int32_t* error_flag);

/* Scratch bytes pa_prefill and pa_prefill_int8 need on the current device, whatever
 * the batch (0 for an invalid head_size). */
size_t pa_prefill_workspace_size(int head_size);

#ifdef __cplusplus
}
#endif

#endif /* PA_PREFILL_H */
