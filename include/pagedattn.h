/*
 * pagedattn.h - C ABI of the GB300 (sm_103a) paged decode-attention library.
 *
 * The operation is the PagedAttention decode step described in "vLLM
 * three-process architecture and the PagedAttention kernel" (devpress.csdn.net),
 * section 3 "PagedAttention 内核原理：从概念到 CUDA 实现":
 *   3.1 "输入是什么": query[num_seqs, num_heads, head_size],
 *       block_tables[num_seqs, max_blocks_per_seq],
 *       k_cache / v_cache[num_physical_blocks, block_size, num_kv_heads, head_size];
 *   3.2 "内核执行流程（简化版）": for each sequence, read its block table (step 1),
 *       derive the number of logical blocks from its valid length (step 2),
 *       gather K/V from the scattered physical blocks (step 3), run standard
 *       attention with the step's query (step 4), write the output (step 5).
 * Section 2 "工作流程拆解", item 4, appends each new token's K/V into the
 * sequence's current physical block: pa_write_cache.
 *
 * Conventions shared by every entry point
 *   - Every tensor pointer is DEVICE memory owned by the caller, dense and
 *     row-major in the shape given.  The library never frees or keeps it.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Calls
 *     are asynchronous on that stream and never synchronise the host, except
 *     where the library's own scratch is allocated, grown or taken over (a
 *     NULL workspace: see pa_decode and pa_decode_mod).
 *   - Calls may be made from several host threads at once, also on one stream
 *     and without a workspace: the library's scratch is held from a call's
 *     lookup until its last launch is queued.
 *   - The return value is PA_OK (0) or a negative PA_ERR_* code, whose cause
 *     pa_last_error() describes; on error nothing was launched (PA_ERR_CUDA
 *     from a launch itself: nothing after that launch).
 *   - `dtype` is PA_F32 or PA_BF16 and applies to query, out, the pools and
 *     the new K/V rows alike.  Arithmetic is fp32 in every case.
 *   - Query head h reads KV head h / (num_heads / num_kv_heads).
 *   - context_lens[s] counts every valid token of sequence s, including the
 *     current step's (written by pa_write_cache first).  Token t of sequence s
 *     is row t % block_size of physical block block_tables[s][t / block_size].
 *     Table entries at or past ceil(context_lens[s] / block_size) are never
 *     read.  Pool rows no valid token occupies never affect the result; the
 *     bf16 and FP8 decode paths do read the unused rows of a sequence's last,
 *     partly filled block (they copy whole runs of rows), so those rows must
 *     lie in the pool, but their contents (even NaN) do not matter.
 *     context_lens[s] == 0 gives an all-zero output row.
 *   - Device-detected input faults (a block id outside [0, num_physical_blocks),
 *     a context length beyond max_blocks_per_seq * block_size or negative, a
 *     slot outside the pool) are reported by OR-ing PA_DEVERR_* bits into the
 *     optional device word `error_flag`; the offending row is skipped (its
 *     content is then unspecified) instead of being read or written.
 *   - Kernels are launched with programmatic stream serialisation: a kernel
 *     may become resident while the one before it on the stream finishes, but
 *     it reads and writes nothing until that kernel has completed
 *     (griddepcontrol.wait).
 */
#ifndef PAGEDATTN_H
#define PAGEDATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define PA_OK 0
#define PA_ERR_INVALID_ARG (-1) /* null pointer, bad size, misaligned pointer */
#define PA_ERR_UNSUPPORTED (-2) /* valid but not built: head_size, group size, dtype */
#define PA_ERR_CUDA (-3)        /* a CUDA runtime call failed (message kept) */
#define PA_ERR_WORKSPACE (-4)   /* caller workspace smaller than required */

/* Element types. */
#define PA_F32 0
#define PA_BF16 1
#define PA_FP8_E4M3 2 /* pool element only: 1 sign, 4 exponent (bias 7), 3 mantissa bits; max 448 */

/* Bits OR-ed into the optional device error word. */
#define PA_DEVERR_BLOCK_ID 1    /* block id outside [0, num_physical_blocks) */
#define PA_DEVERR_CONTEXT_LEN 2 /* context length < 0 or > max_blocks_per_seq*block_size (clamped) */
#define PA_DEVERR_SLOT 4        /* slot_mapping entry >= num_physical_blocks*block_size (skipped) */
#define PA_DEVERR_TIMEOUT 8     /* a pipeline wait exceeded its limit; the kernel returned early */
#define PA_DEVERR_STATE 32      /* a kernel found its own bookkeeping wrong, used none of it and returned early (16: pa_tables.h) */

/*
 * pa_decode - paged decode attention, one query token per sequence.
 *
 *   out[s, h, :] = sum_t softmax_t(scale * <query[s, h, :], K_s[t, h/G, :]>) V_s[t, h/G, :]
 *
 * out          [num_seqs, num_heads, head_size], dtype            (written)
 * query        [num_seqs, num_heads, head_size], dtype
 * k_cache      [num_physical_blocks, block_size, num_kv_heads, head_size], dtype
 * v_cache      same shape as k_cache
 * block_tables [num_seqs, max_blocks_per_seq] int32
 * context_lens [num_seqs] int32
 * Requirements: num_heads % num_kv_heads == 0 and num_heads / num_kv_heads <= 8;
 * head_size 64 or 128; block_size in [1, 4096]; query, out and both pools
 * 16-byte aligned; for bf16, fewer than 2^31 token rows in the pool
 * (num_physical_blocks * block_size) else PA_ERR_UNSUPPORTED.
 * bf16 pools are read through TMA tensor maps built on the host for each call
 * (cuTensorMapEncodeTiled, taken from the driver; PA_ERR_CUDA if the driver
 * lacks it); block sizes that are multiples of 8 stream fastest.
 * The batch's tiles of 16 tokens are split into equal ranges, one CTA each.
 * A sequence cut by range boundaries leaves partial softmax statistics per
 * range; the last CTA to finish one of its KV heads merges them by
 * log-sum-exp in a second pass over the partials.  The scratch for that comes
 * from a per-device buffer the library allocates (zero-filled) on first use
 * and grows when a larger batch needs it (cudaMalloc, which synchronises the
 * device; use pa_decode_ws to supply the scratch and never allocate).  That
 * buffer is shared by every call on the device: calls that may run at the
 * same time on different streams must use pa_decode_ws with scratch of their
 * own, and so must a graph that may run beside other calls.  (The buffer a
 * captured call has taken is not freed when a larger batch needs another.)
 */
int pa_decode(void* out, const void* query, const void* k_cache, const void* v_cache,
              const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
              int num_heads, int num_kv_heads, int head_size, int block_size,
              int max_blocks_per_seq, float scale, void* stream, int dtype);

/*
 * pa_decode_workspace_size - bytes of scratch pa_decode_ws needs on the
 * current device for this batch shape (num_ranges as in pa_decode_ex; 0 =
 * the default of one range per SM).  Returns 0 for invalid sizes.
 */
size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                                int num_ranges);

/*
 * pa_decode_ws - pa_decode with caller-owned scratch (device memory of at
 * least pa_decode_workspace_size(...) bytes, 256-byte aligned).  Never
 * allocates.  The scratch must be zero-filled before its first use; every
 * call that completes leaves it zero-filled again, so it can be reused by the
 * next call on the same stream.  Two calls that overlap in time must not
 * share it.  After a call that reported PA_DEVERR_TIMEOUT, zero it again.
 */
int pa_decode_ws(void* out, const void* query, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                 int num_heads, int num_kv_heads, int head_size, int block_size,
                 int max_blocks_per_seq, float scale, void* stream, int dtype, void* workspace,
                 size_t workspace_bytes);

/*
 * pa_decode_ex - the general form behind pa_decode and pa_decode_ws.
 *
 * num_physical_blocks  > 0: every block id read from block_tables is checked
 *                      against it on the device (PA_DEVERR_BLOCK_ID); 0: unchecked
 *                      (bf16 and FP8 pools must then lie in memory that the driver
 *                      knows the extent of: rows beyond the allocation read as
 *                      zeros; PA_ERR_INVALID_ARG if it does not).  Give the size of
 *                      pools in a reserved address range that is mapped in part:
 *                      the extent known there is the whole range.
 * workspace            NULL: library-owned scratch (may allocate, see pa_decode).
 * num_ranges           0: one token range per SM (the default).  > 0: split the
 *                      flattened batch into exactly this many ranges (1 = a
 *                      single CTA walks every sequence in one pass).
 * error_flag           optional device int32 that receives PA_DEVERR_* bits.
 */
int pa_decode_ex(void* out, const void* query, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                 int num_heads, int num_kv_heads, int head_size, int block_size,
                 int max_blocks_per_seq, float scale, void* stream, int dtype,
                 int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                 int32_t* error_flag);

/*
 * pa_decode_append - one decode step with its cache write fused in: for every
 * sequence s with context_lens[s] >= 1, the K/V of its newest token (position
 * context_lens[s] - 1) are k_new[s] / v_new[s]; the call stores them into the
 * pool at that position (block_tables[s][(c-1) / block_size], row
 * (c-1) % block_size) and returns the same `out` as pa_write_cache of those
 * rows followed by pa_decode_ex.  One launch instead of two: the decode
 * itself puts the new rows into its staged tile and into the pool.
 * k_new, v_new  [num_seqs, num_kv_heads, head_size], 16-byte aligned
 * The newest token's block must not be shared with another sequence of the
 * batch (copy-on-write first, as pa_bm_append arranges).  dtype PA_BF16 only
 * (PA_ERR_UNSUPPORTED otherwise; FP8 pools: pa_decode_fp8_append).  Other arguments as in pa_decode_ex; a
 * failed block-id check (num_physical_blocks > 0) leaves that token unwritten.
 */
int pa_decode_append(void* out, const void* query, const void* k_new, const void* v_new,
                     void* k_cache, void* v_cache, const int32_t* block_tables,
                     const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                     int head_size, int block_size, int max_blocks_per_seq, float scale,
                     void* stream, int dtype, int num_physical_blocks, void* workspace,
                     size_t workspace_bytes, int num_ranges, int32_t* error_flag);

/*
 * pa_decode_mq - several query tokens per sequence over the paged cache, with
 * a causal mask: the chunked-prefill / speculative-decoding-verification step
 * (named by the vLLM book preface's reader questions and the is96 essay's
 * feature list) built on the same gather as pa_decode.
 *
 *   out[s, i, h, :] = attention of query[s, i, h, :] over the keys/values at
 *                     positions 0 .. context_lens[s] - num_queries + i
 *
 * query, out  [num_seqs, num_queries, num_heads, head_size]
 * The num_queries newest tokens of every sequence must already be in the pool
 * (pa_write_cache) and counted in context_lens.  A query whose position is
 * negative (context shorter than num_queries) gets a zero row.
 * Requires dtype PA_BF16 and (num_heads / num_kv_heads) * num_queries <= 32;
 * num_queries == 1 is plain decode.  Other arguments as in pa_decode_ex; the
 * scratch size comes from pa_decode_mq_workspace_size (workspace NULL: the
 * library's own, allocated on first use).
 */
int pa_decode_mq(void* out, const void* query, const void* k_cache, const void* v_cache,
                 const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                 int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                 int max_blocks_per_seq, float scale, void* stream, int dtype,
                 int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                 int32_t* error_flag);

/* Scratch bytes pa_decode_mq needs (0 for invalid sizes). */
size_t pa_decode_mq_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                   int head_size, int num_ranges);

/*
 * pa_decode_mq_append - pa_decode_mq with the step's cache write fused in: for
 * every sequence s with context c = context_lens[s], the K/V of its query
 * token i (position c - num_queries + i) are k_new[s * num_queries + i] /
 * v_new[s * num_queries + i]; the call stores each token whose position is
 * >= 0 into the pool (block_tables[s][pos / block_size], row
 * pos % block_size) and returns the same `out` as pa_write_cache of those
 * rows followed by pa_decode_mq.  One launch instead of two when
 * (num_heads / num_kv_heads) * num_queries <= 8; above that (two to four
 * consumer warps per KV head) the call launches a row-writing kernel and then the
 * decode on `stream`, chained by programmatic dependent launch.
 * k_new, v_new  [num_seqs * num_queries, num_kv_heads, head_size], bf16,
 *               16-byte aligned
 * The blocks of the new tokens must not be shared with another sequence of
 * the batch.  dtype PA_BF16 only (PA_ERR_UNSUPPORTED otherwise).  Other
 * arguments, scratch size and limits as in pa_decode_mq; a failed block-id
 * check (num_physical_blocks > 0) leaves that token unwritten.
 */
int pa_decode_mq_append(void* out, const void* query, const void* k_new, const void* v_new,
                        void* k_cache, void* v_cache, const int32_t* block_tables,
                        const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                        int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq,
                        float scale, void* stream, int dtype, int num_physical_blocks,
                        void* workspace, size_t workspace_bytes, int num_ranges,
                        int32_t* error_flag);

/*
 * pa_decode_mod - decode with modified scores, one or several query tokens
 * per sequence: the masks and biases models put on the same gather as
 * pa_decode_mq.  With pos = context_lens[s] - num_queries + i the position of
 * query i and c = context_lens[s], token t of sequence s has the score
 *
 *   score = softcap * tanh(scale * <q, k_t> / softcap) - alibi_slopes[h] * |pos - t|
 *
 * (softcap 0: scale * <q, k_t>; alibi_slopes NULL: no distance term), and query i
 * sees it if 0 <= pos, t < c, t >= first_tokens[s], and
 *
 *   t < prefix_lens[s]   or   ( t <= pos  and  (window == 0 or pos - t < window) )
 *
 * softcap      >= 0, finite (tanh cap of the scores; 0: none)
 * alibi_slopes [num_heads] float or NULL (finite, also times a distance)
 * window       >= 0: tokens a query sees back, its own included (0: all)
 * first_tokens [num_seqs] int32 or NULL: first token a sequence's queries see
 *              (the start of their document); below 0 counts as 0
 * prefix_lens  [num_seqs] int32 or NULL: tokens before this one are seen by every
 *              query, also behind its position and its window (a
 *              bidirectional prefix, or first tokens kept in sight); clamped
 *              to [0, context_lens[s]]
 * query, out   [num_seqs, num_queries, num_heads, head_size]
 * A query that sees nothing gets a zero row.  Tokens no query of their sequence
 * sees are not attended whatever the pool holds there (even NaN), and the table
 * entries of blocks without a seen token may be stale: the blocks a window has
 * left behind can be freed.  A token that some query of the sequence sees must
 * be finite for the others too.
 * Types: PA_F32 (num_queries == 1) or PA_BF16; (num_heads / num_kv_heads) *
 * num_queries <= 32.
 * workspace    256-byte aligned device scratch of at least
 *              pa_decode_mod_workspace_size(...) bytes, of any content; two calls
 *              that may overlap in time must not share it.  NULL: the library's
 *              own, one buffer per stream, refused while `stream` is being
 *              captured (PA_ERR_INVALID_ARG).  It is allocated at a stream's first
 *              call and when a batch outgrows it; those calls, and a first call
 *              on a ninth stream, which takes over the buffer used longest ago,
 *              may wait for the device.
 * Other arguments as in pa_decode_mq.  The call makes two launches: the walk, and
 * a merge of the sequences that range boundaries cut.
 *
 * pa_decode_fp8_mod - the same over FP8 pools: keys and values as in
 * pa_decode_fp8, query and out bf16.
 */
int pa_decode_mod(void* out, const void* query, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                  int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                  int max_blocks_per_seq, float scale, float softcap, const float* alibi_slopes,
                  int window, const int32_t* first_tokens, const int32_t* prefix_lens, void* stream,
                  int dtype, int num_physical_blocks, void* workspace, size_t workspace_bytes,
                  int num_ranges, int32_t* error_flag);
int pa_decode_fp8_mod(void* out, const void* query, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                      int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                      int max_blocks_per_seq, float scale, float k_scale, float v_scale, float softcap,
                      const float* alibi_slopes, int window, const int32_t* first_tokens,
                      const int32_t* prefix_lens, void* stream, int num_physical_blocks, void* workspace,
                      size_t workspace_bytes, int num_ranges, int32_t* error_flag);

/* Scratch bytes pa_decode_mod (kv_dtype PA_F32 or PA_BF16) or pa_decode_fp8_mod
 * (PA_FP8_E4M3) needs on the current device (0 for invalid sizes). */
size_t pa_decode_mod_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                    int head_size, int kv_dtype, int num_ranges);

/*
 * pa_decode_prefix - pa_decode_mq for a batch whose sequences share a long
 * prefix (a system prompt, a document, samples of one prompt), attended once
 * for all of them: the prefix's K/V are read once per call instead of once per
 * sequence, and its scores are one matrix product per KV head.
 *
 * prefix_table [num_prefix_blocks] int32: the physical blocks of the prefix's
 *              P = num_prefix_blocks * block_size tokens (may be NULL for 0)
 * block_tables [num_seqs, max_blocks_per_seq]: the sequences' whole tables, as
 *              for pa_decode_mq
 * A sequence of context_lens[s] >= P + num_queries - 1 tokens has the prefix as its
 * first P tokens; the entries of its row before num_prefix_blocks are not read.
 * A shorter one (a padding row of context 0, a request that has not reached the
 * end of the prompt) is attended through its own row alone.  So out is that of
 * pa_decode_mq wherever the rows of the longer sequences begin with
 * prefix_table, as pa_bm_share_prefix and pa_tables_step make them.
 * Requires PA_BF16; block_size a multiple of 8 (PA_ERR_UNSUPPORTED otherwise);
 * num_prefix_blocks <= max_blocks_per_seq; (num_heads / num_kv_heads) *
 * num_queries <= 32.  num_physical_blocks > 0 checks the prefix's block ids
 * too; tokens of a bad one count as zeros.
 * With more than 128 query rows per KV head (num_seqs * num_queries * group) the
 * softmax weights of the prefix enter its second product rounded to bf16
 * (relative error <= 2^-8 each), with fewer to about 2^-16; sums and statistics
 * stay fp32.
 * workspace    256-byte aligned device scratch of at least
 *              pa_decode_prefix_workspace_size(...) bytes; or NULL: as in
 *              pa_decode_mod
 * Other arguments as in pa_decode_mq.  The call makes up to three launches.
 *
 * pa_decode_fp8_prefix - the same over FP8 pools: keys, values and the query's
 * rounding as in pa_decode_fp8_mq, query and out bf16.  The softmax weights of
 * the prefix enter its second product rounded to f16: off by at most 2^-11 of
 * themselves or 2^-32 of the largest, whichever is more.  head_size 64 with an
 * odd num_kv_heads is PA_ERR_UNSUPPORTED.
 */
int pa_decode_prefix(void* out, const void* query, const void* k_cache, const void* v_cache,
                     const int32_t* prefix_table, const int32_t* block_tables,
                     const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                     int num_kv_heads, int head_size, int block_size, int num_prefix_blocks,
                     int max_blocks_per_seq, float scale, void* stream, int dtype,
                     int num_physical_blocks, void* workspace, size_t workspace_bytes,
                     int32_t* error_flag);

int pa_decode_fp8_prefix(void* out, const void* query, const void* k_cache, const void* v_cache,
                         const int32_t* prefix_table, const int32_t* block_tables,
                         const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                         int num_kv_heads, int head_size, int block_size, int num_prefix_blocks,
                         int max_blocks_per_seq, float scale, float k_scale, float v_scale, void* stream,
                         int num_physical_blocks, void* workspace, size_t workspace_bytes,
                         int32_t* error_flag);

/* Scratch bytes pa_decode_prefix or pa_decode_fp8_prefix needs on the current device (0 for invalid sizes). */
size_t pa_decode_prefix_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                       int head_size);

/*
 * pa_write_cache - scatter one step's new K/V rows into the paged pool
 * (the "reshape_and_cache" step).  For every token i with slot_mapping[i] >= 0:
 *   k_cache[slot / block_size, slot % block_size, :, :] = k_new[i, :, :]  (bit copy)
 * and the same for V.  Negative slots are padding and are skipped; slots at
 * or beyond num_physical_blocks * block_size are skipped and reported.
 * Duplicate slots within one call leave either row (unspecified which).
 * k_new, v_new  [num_tokens, num_kv_heads, head_size], dtype, 16-byte aligned
 * slot_mapping  [num_tokens] int64
 * k_cache, v_cache as in pa_decode (written in place).
 */
int pa_write_cache(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                   void* k_cache, void* v_cache, int num_tokens, int num_kv_heads, int head_size,
                   int block_size, int num_physical_blocks, void* stream, int dtype);

/* pa_write_cache_ex - pa_write_cache with an optional device error word. */
int pa_write_cache_ex(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                      void* k_cache, void* v_cache, int num_tokens, int num_kv_heads,
                      int head_size, int block_size, int num_physical_blocks, void* stream,
                      int dtype, int32_t* error_flag);

/*
 * pa_decode_static - pa_decode for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this entry point; it exists for callers
 * that cannot call cudaMalloc when they decode, e.g. a serving engine whose
 * own allocator has already reserved nearly all device memory, or a latency
 * path that cannot afford cudaMalloc's implicit device synchronisation.
 * Arguments, layouts and results are those of pa_decode.  Instead of
 * allocating scratch it uses an array of PA_STATIC_SCRATCH_BYTES compiled
 * into the library: every GPU that loads the library holds that memory until
 * the process exits.  Nothing is allocated or freed by this call.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current); make that first call
 *     before any stream capture.
 *   - Arguments are checked as pa_decode checks them, with the same return
 *     codes; a rejected call queues nothing on `stream`.
 *   - All calls share the one array, which keeps the previous call's
 *     contents; each accepted call clears the part that must start at zero
 *     (cudaMemsetAsync on `stream`) right before its kernel.  Calls that
 *     overlap in time on the GPU (different streams, no ordering) race on
 *     the array.
 *   - Batches whose scratch exceeds PA_STATIC_SCRATCH_BYTES are rejected with
 *     PA_ERR_WORKSPACE before anything is queued (the scratch is at most
 *     pa_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, 0)
 *     bytes: about 5 MB for 64 sequences of 32 query / 8 KV heads of 128).
 */
#define PA_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)
int pa_decode_static(void* out, const void* query, const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                     int num_heads, int num_kv_heads, int head_size, int block_size,
                     int max_blocks_per_seq, float scale, void* stream, int dtype);

/*
 * FP8 KV pool.  The pages list quantisation among vLLM's features but give no
 * format; this library's reading: the pool holds E4M3 codes with one float
 * scale per pool (k_scale, v_scale), a code c standing for e4m3(c) * scale.
 *
 * pa_write_cache_fp8 - pa_write_cache into FP8 pools: each new element x
 * becomes the E4M3 code nearest to x / scale (the quotient in float32, ties to
 * even, saturating at +-448).  k_new/v_new are PA_BF16 or PA_F32 (src_dtype);
 * k_cache/v_cache are uint8 [num_physical_blocks, block_size, num_kv_heads,
 * head_size].  error_flag as in pa_write_cache_ex (optional).
 *
 * pa_decode_fp8 - pa_decode_ex over FP8 pools (one query per sequence; several:
 * pa_decode_fp8_mq), query and out bf16: scores use
 * k = e4m3(code) * k_scale and values v = e4m3(code) * v_scale.  Each token
 * moves half the bytes of a bf16 pool.  Scratch as pa_decode_workspace_size.
 * The query is rounded to f16 on the way into the tensor cores (exact for
 * |q| in [2^-14, 65504]), and so are the softmax weights: off by at most 2^-11
 * of themselves or 2^-39 of the largest, whichever is more.  head_size 64 with
 * an odd num_kv_heads is PA_ERR_UNSUPPORTED (a KV-head group's FP8 row must be
 * whole 128-byte lines).
 */
int pa_write_cache_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                       void* k_cache, void* v_cache, int num_tokens, int num_kv_heads, int head_size,
                       int block_size, int num_physical_blocks, float k_scale, float v_scale,
                       void* stream, int src_dtype, int32_t* error_flag);
int pa_decode_fp8(void* out, const void* query, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                  int num_heads, int num_kv_heads, int head_size, int block_size,
                  int max_blocks_per_seq, float scale, float k_scale, float v_scale, void* stream,
                  int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                  int32_t* error_flag);

/*
 * pa_decode_fp8_append - pa_decode_append over FP8 pools: the newest token's
 * bf16 K/V (k_new/v_new [num_seqs, num_kv_heads, head_size]) are quantised
 * as pa_write_cache_fp8 does (bit-identical codes) and written into the pools
 * by the decode launch itself; out equals pa_write_cache_fp8 followed by
 * pa_decode_fp8.  Scales, layouts and limits as in pa_decode_fp8.
 */
int pa_decode_fp8_append(void* out, const void* query, const void* k_new, const void* v_new,
                         void* k_cache, void* v_cache, const int32_t* block_tables,
                         const int32_t* context_lens, int num_seqs, int num_heads, int num_kv_heads,
                         int head_size, int block_size, int max_blocks_per_seq, float scale,
                         float k_scale, float v_scale, void* stream, int num_physical_blocks,
                         void* workspace, size_t workspace_bytes, int num_ranges, int32_t* error_flag);

/*
 * pa_decode_fp8_mq - pa_decode_mq over FP8 pools: several causal query tokens
 * per sequence (chunked prefill, speculative-decoding verification) reading
 * the quantised cache.  Keys and values are e4m3(code) * k_scale and
 * e4m3(code) * v_scale as in pa_decode_fp8; query and out are bf16
 * [num_seqs, num_queries, num_heads, head_size]; query i of sequence s sees
 * positions 0 .. context_lens[s] - num_queries + i.  Requires
 * (num_heads / num_kv_heads) * num_queries <= 32.  Scratch size:
 * pa_decode_mq_workspace_size.  Other arguments and limits as in
 * pa_decode_fp8 and pa_decode_mq.
 *
 * pa_decode_fp8_mq_append - the same with the step's quantising cache write
 * fused in: k_new / v_new [num_seqs * num_queries, num_kv_heads, head_size]
 * bf16 (row s * num_queries + i: position context_lens[s] - num_queries + i)
 * are quantised as pa_write_cache_fp8 does (bit-identical codes) and stored
 * into the pools; tokens at negative positions are skipped.  Up to 8
 * (query, head) columns per KV head the decode launch itself writes them;
 * above that a row-writing kernel is chained ahead of the decode.  out equals
 * pa_write_cache_fp8 of those rows followed by pa_decode_fp8_mq.
 */
int pa_decode_fp8_mq(void* out, const void* query, const void* k_cache, const void* v_cache,
                     const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                     int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                     int max_blocks_per_seq, float scale, float k_scale, float v_scale, void* stream,
                     int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                     int32_t* error_flag);
int pa_decode_fp8_mq_append(void* out, const void* query, const void* k_new, const void* v_new,
                            void* k_cache, void* v_cache, const int32_t* block_tables,
                            const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                            int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq,
                            float scale, float k_scale, float v_scale, void* stream,
                            int num_physical_blocks, void* workspace, size_t workspace_bytes,
                            int num_ranges, int32_t* error_flag);

/*
 * pa_test_stall_copy - test hook for the decode kernel's bounded waits; the
 * pages have no counterpart.  Every wait of the decode pipeline (a consumer
 * waiting for a stage's copies, the copy engine's issuer waiting for a free
 * stage) gives up after a time limit, sets PA_DEVERR_TIMEOUT in error_flag and
 * ends the kernel early, so that a copy that never lands cannot hang the GPU.
 * This hook lets a test reach that path without any fault: the next decode
 * call on the calling thread that launches its kernel (pa_decode*, any
 * variant) withholds every copy of flattened tile `tile` (the batch's tiles of
 * 16 tokens, sequence after sequence, counted from 0) and bounds every wait by
 * wait_limit_us microseconds (0: the default of 2 s).  The stage meant for
 * that tile is never filled, the waits on it run out, and the kernel returns
 * after letting the copies it had started land (again within the limit).
 * (pa_decode_prefix: its prefix kernel, whose tiles of 128 prefix tokens are
 * counted per KV head and per 256 query rows of it, one after another, and behind
 * them the tiles of the walk behind the prefix; pa_decode_mod: the tiles its walk takes.)
 * That call's output is unspecified, and its scratch (pa_decode_ws) must be
 * zero-filled again before reuse.  The setting is used by one launch and then
 * cleared; tile = -1 clears it.  Returns PA_OK, or PA_ERR_INVALID_ARG for
 * tile < -1.
 */
int pa_test_stall_copy(long long tile, unsigned int wait_limit_us);

/* Message for the calling thread's last non-zero return ("" if none). */
const char* pa_last_error(void);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_H */
