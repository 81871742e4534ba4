// Decode with modified scores (pa_decode_mod, pa_decode_fp8_mod): the decode
// kernel with kWalkMod.
//
//   s_t = cap * tanh(scale * <q, k_t> / cap) - slope_h * |pos - t|
//   t is seen: t < c, t >= first and (t < prefix or pos - window < t <= pos)
//
// As plain decode it is bound by the K/V bytes, so the walk leaves out the tiles
// that no query of a sequence sees: per sequence the tiles of [first, prefix),
// then those from the first query's window on (SeqWalk), both cut into the same
// equal ranges.  Inside a tile, rows nobody sees are neither copied (whole boxes)
// nor used (their scores are -inf and their V entries zeroed in registers).
#include "pa_launch.cuh"

#include <cmath>

#include "pa_decode_impl.h"

namespace pa {

int launch_mod(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool f32,
               bool kv_fp8) {
  const bool wide = prm.group * prm.num_queries > 8;  // two to four warps per KV head
  if (f32) {
    if (head_size == 64)
      return prm.group <= 2 ? launch_typed<float, 64, 2, 0, false, kWalkMod>(prm, pl, dev, stream)
                            : launch_typed<float, 64, 8, 0, false, kWalkMod>(prm, pl, dev, stream);
    if (prm.group <= 2) return launch_typed<float, 128, 2, 0, false, kWalkMod>(prm, pl, dev, stream);
    return prm.group <= 4 ? launch_typed<float, 128, 4, 0, false, kWalkMod>(prm, pl, dev, stream)
                          : launch_typed<float, 128, 8, 0, false, kWalkMod>(prm, pl, dev, stream);
  }
  using T = __nv_bfloat16;
  if (head_size == 64) {
    if (kv_fp8)
      return wide ? launch_typed<T, 64, 8, 2, true, kWalkMod>(prm, pl, dev, stream)
                  : launch_typed<T, 64, 8, 1, true, kWalkMod>(prm, pl, dev, stream);
    return wide ? launch_typed<T, 64, 8, 2, false, kWalkMod>(prm, pl, dev, stream)
                : launch_typed<T, 64, 8, 1, false, kWalkMod>(prm, pl, dev, stream);
  }
  if (kv_fp8)
    return wide ? launch_typed<T, 128, 8, 2, true, kWalkMod>(prm, pl, dev, stream)
                : launch_typed<T, 128, 8, 1, true, kWalkMod>(prm, pl, dev, stream);
  return wide ? launch_typed<T, 128, 8, 2, false, kWalkMod>(prm, pl, dev, stream)
              : launch_typed<T, 128, 8, 1, false, kWalkMod>(prm, pl, dev, stream);
}

namespace {

int make_extras(DecodeExtras* ex, float softcap, const float* alibi_slopes, int window,
                const int32_t* first_tokens, const int32_t* prefix_lens) {
  clear_error();
  if (!std::isfinite(softcap) || softcap < 0.f)
    return fail(PA_ERR_INVALID_ARG, "pa_decode_mod: softcap must be finite and not negative (0: none)");
  if (window < 0) return fail(PA_ERR_INVALID_ARG, "pa_decode_mod: window %d < 0 (0: none)", window);
  if (!aligned(alibi_slopes, 4) || !aligned(first_tokens, 4) || !aligned(prefix_lens, 4))
    return fail(PA_ERR_INVALID_ARG, "pa_decode_mod: misaligned tensor pointer");
  ex->walk = kWalkMod;
  ex->softcap = softcap;
  ex->alibi_slopes = alibi_slopes;
  ex->window = window;
  ex->first_tokens = first_tokens;
  ex->prefix_lens = prefix_lens;
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" int pa_decode_mod(void* out, const void* query, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                             int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                             int max_blocks_per_seq, float scale, float softcap, const float* alibi_slopes,
                             int window, const int32_t* first_tokens, const int32_t* prefix_lens, void* stream,
                             int dtype, int num_physical_blocks, void* workspace, size_t workspace_bytes,
                             int num_ranges, int32_t* error_flag) {
  pa::DecodeExtras ex{};
  const int rc = pa::make_extras(&ex, softcap, alibi_slopes, window, first_tokens, prefix_lens);
  if (rc != PA_OK) return rc;
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, stream,
                           dtype, num_physical_blocks, workspace, workspace_bytes, num_ranges, error_flag, false,
                           1.f, 1.f, nullptr, nullptr, nullptr, &ex);
}

extern "C" int pa_decode_fp8_mod(void* out, const void* query, const void* k_cache, const void* v_cache,
                                 const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                                 int num_queries, int num_heads, int num_kv_heads, int head_size,
                                 int block_size, int max_blocks_per_seq, float scale, float k_scale,
                                 float v_scale, float softcap, const float* alibi_slopes, int window,
                                 const int32_t* first_tokens, const int32_t* prefix_lens, void* stream,
                                 int num_physical_blocks, void* workspace, size_t workspace_bytes,
                                 int num_ranges, int32_t* error_flag) {
  pa::DecodeExtras ex{};
  const int rc = pa::make_extras(&ex, softcap, alibi_slopes, window, first_tokens, prefix_lens);
  if (rc != PA_OK) return rc;
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, stream,
                           PA_BF16, num_physical_blocks, workspace, workspace_bytes, num_ranges, error_flag, true,
                           k_scale, v_scale, nullptr, nullptr, nullptr, &ex);
}
