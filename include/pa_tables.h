/*
 * pa_tables.h - one step's block tables and slot map, built on the GPU (C ABI).
 *
 * The device counterpart of pa_block_manager.h for engines that keep the
 * lengths of their requests on the GPU: "vLLM three-process architecture and
 * the PagedAttention kernel" (devpress.csdn.net), section 1.2 (free pool of
 * blocks, block table per sequence) and section 2 item 4 (a new token gets a new
 * block when the current one is full).  A whole step (tables, cache write,
 * decode) then runs, and can be captured, without the host seeing a length.
 *
 * Conventions are those of pagedattn.h: device pointers owned by the caller,
 * asynchronous on `stream`, PA_OK or a negative PA_ERR_* code with a message
 * in pa_last_error(), nothing queued on error.
 */
#ifndef PA_TABLES_H
#define PA_TABLES_H

#include <stdint.h>

#include "pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_TABLES_RELEASE (-1) /* new_lens entry: the sequence gives its blocks back */

/* Bit OR-ed into error_flag beside those of pagedattn.h. */
#define PA_DEVERR_NO_BLOCKS 16 /* the free list cannot supply a sequence's blocks; it is not served */

/*
 * pa_tables_step - one step's growth and release of a batch of sequences.
 *
 * For every sequence s, in order, new_lens[s] says what happens to it:
 *   n > 0  it gets n tokens.  A sequence with context 0 starts: its first
 *          num_prefix_blocks table entries become prefix_table and its
 *          context num_prefix_blocks * block_size before the new tokens.  Blocks
 *          that the new tokens need are taken from the end of the free list and
 *          entered in its row of block_tables.
 *   n = 0  nothing.
 *   n = PA_TABLES_RELEASE  its own blocks (table entries num_prefix_blocks ..
 *          ceil(context / block_size) - 1, never the prefix's) are put at the
 *          end of the free list, in table order, and its context becomes 0.
 *          Its row is left as it is.  All releases come before the first block
 *          is taken, so a step's returned blocks serve the same step.
 *
 * block_tables     [num_seqs, max_blocks_per_seq] int32, entries entered in place
 * context_lens_out [num_seqs] int32: the lengths after the step
 * seq_starts       [num_seqs + 1] int32: tokens of the sequences before s (the
 *                  last entry: all tokens of the step)
 * slot_mapping     [max_tokens] int64: slots of the new tokens, sequence after
 *                  sequence (entry seq_starts[s] + i: token i of sequence s),
 *                  as pa_write_cache reads them; -1 behind the last token
 * free_blocks      [num_physical_blocks] int32: the free list, a stack whose
 *                  free_count first entries are free blocks (in place)
 * free_count_out   [1] int32: its length after the step
 * context_lens     [num_seqs] int32, new_lens [num_seqs] int32, free_count [1]
 *                  int32: before the step
 * prefix_table     [num_prefix_blocks] int32 (may be NULL for 0): blocks of the
 *                  prefix that all sequences of these tables share
 * error_flag       optional device int32 that receives PA_DEVERR_* bits
 *
 * A sequence is served whole or not at all.  One whose new length does not fit
 * its row (PA_DEVERR_CONTEXT_LEN) is left as it is and the others go on.  Once
 * the free list (PA_DEVERR_NO_BLOCKS) or max_tokens (PA_DEVERR_SLOT) cannot
 * hold a sequence, it and every later one that asks for tokens keep their
 * lengths and get no slots.  Lengths below 0, beyond the row or inside the
 * prefix, and new_lens below -1, leave their sequence as it is
 * (PA_DEVERR_CONTEXT_LEN).  A free_count outside [0, num_physical_blocks] is
 * clamped, and blocks returned beyond num_physical_blocks are dropped
 * (PA_DEVERR_BLOCK_ID).  Block ids themselves are passed on unchecked.
 * No output may overlap an input or another output (PA_ERR_INVALID_ARG): a loop
 * keeps two buffers for the lengths and the count and swaps them.  Because the
 * inputs stay, a step repeated on the same inputs gives the same outputs.
 * At most 12288 sequences, block_size at most 4096 (PA_ERR_UNSUPPORTED).
 */
int pa_tables_step(int32_t* block_tables, int32_t* context_lens_out, int32_t* seq_starts,
                   int64_t* slot_mapping, int32_t* free_blocks, int32_t* free_count_out,
                   const int32_t* context_lens, const int32_t* new_lens, const int32_t* free_count,
                   const int32_t* prefix_table, int num_prefix_blocks, int num_seqs,
                   int max_blocks_per_seq, int block_size, int num_physical_blocks, int max_tokens,
                   void* stream, int32_t* error_flag);

#ifdef __cplusplus
}
#endif

#endif /* PA_TABLES_H */
