// Decode over int8 pools (pa_decode_int8): the decode kernel's walk with codes widened to
// f16 and the tokens' scales beside them in every stage; shapes that it does not take run as
// chunks (pa_prefill.cu).  Integers up to 127 are f16 numbers; scores and weights take the
// scales in fp32.  64 sequences of 512 to 4,096: 64.5 us (217 as chunks, whose 128 rows one token hardly
// fills), 4.8 TB/s of codes and scales; 8 of 32k: 106 us (292), 5.1 TB/s.  DRAM is at 58%
// and issue slots at 38%: the copies' latency, and start and end of the launch.  Without the
// scales' copies, 3% of the bytes, 61.7 and 100 us.
#include "pa_chunk.cuh"
#include "pa_decode_impl.h"

namespace pa {

int launch_int8(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size) {
  using T = __nv_bfloat16;
  const int columns = prm.group * prm.num_queries;
  if (head_size == 64) {
    if (prm.num_queries == 1) return launch_typed<T, 64, 8, 0, true, kWalkAll, true>(prm, pl, dev, stream);
    return columns <= 8 ? launch_typed<T, 64, 8, 1, true, kWalkAll, true>(prm, pl, dev, stream)
                        : launch_typed<T, 64, 8, 2, true, kWalkAll, true>(prm, pl, dev, stream);
  }
  if (prm.num_queries == 1) return launch_typed<T, 128, 8, 0, true, kWalkAll, true>(prm, pl, dev, stream);
  return columns <= 8 ? launch_typed<T, 128, 8, 1, true, kWalkAll, true>(prm, pl, dev, stream)
                      : launch_typed<T, 128, 8, 2, true, kWalkAll, true>(prm, pl, dev, stream);
}

namespace {

// Whether the decode kernel has no plan for the shape: more than 32 columns per KV
// head, or rows that are not whole 128-byte lines.
bool runs_as_chunks(int num_queries, int num_heads, int num_kv_heads, int head_size) {
  return (long long)(num_heads / num_kv_heads) * num_queries > kMaxColumns ||
         (long long)num_kv_heads * head_size % kLine != 0;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_int8_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                                int head_size, int num_ranges) {
  using namespace pa;
  if (num_seqs <= 0 || num_queries <= 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      (head_size != 64 && head_size != 128) || num_ranges < 0)
    return 0;
  if (!runs_as_chunks(num_queries, num_heads, num_kv_heads, head_size))
    return decode_workspace_size_q(num_seqs, num_heads, num_kv_heads, head_size, num_ranges, num_queries);
  return pa_prefill_workspace_size(head_size);
}

extern "C" int pa_decode_int8(void* out, const void* query, const void* k_cache, const void* v_cache,
                              const float* k_scales, const float* v_scales, const int32_t* block_tables,
                              const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                              int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq, float scale,
                              void* stream, int num_physical_blocks, void* workspace, size_t workspace_bytes,
                              int num_ranges, int32_t* error_flag) {
  using namespace pa;
  clear_error();
  if (num_queries < 1) return fail(PA_ERR_INVALID_ARG, "pa_decode_int8: num_queries %d < 1", num_queries);
  ChunkCall c{};
  c.int8 = true, c.k_scales = k_scales, c.v_scales = v_scales;
  c.out = out, c.query = query, c.k_cache = k_cache, c.v_cache = v_cache;
  c.block_tables = block_tables, c.context_lens = context_lens;
  c.num_queries = num_queries, c.num_seqs = num_seqs, c.num_heads = num_heads, c.num_kv_heads = num_kv_heads;
  c.head_size = head_size, c.block_size = block_size, c.max_blocks_per_seq = max_blocks_per_seq;
  c.scale = scale, c.stream = stream, c.dtype = PA_BF16, c.num_physical_blocks = num_physical_blocks;
  c.error_flag = error_flag;
  const int rc = prefill_validate(c);
  if (rc != PA_OK) return rc;
  if (num_ranges < 0) return fail(PA_ERR_INVALID_ARG, "pa_decode_int8: num_ranges %d", num_ranges);
  if (runs_as_chunks(num_queries, num_heads, num_kv_heads, head_size)) {
    c.workspace = workspace, c.workspace_bytes = workspace_bytes;
    return prefill_impl(c);
  }
  const TokenScales scales{k_scales, v_scales};
  return decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries, num_heads,
                       num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, stream, PA_BF16,
                       num_physical_blocks, workspace, workspace_bytes, num_ranges, error_flag, true, 1.f, 1.f, nullptr,
                       nullptr, nullptr, nullptr, &scales);
}
