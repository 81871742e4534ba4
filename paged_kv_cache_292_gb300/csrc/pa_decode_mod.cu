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
//
// Measured (HBM copies run at 6.77 TB/s): 64 sequences of 512 to 8192 tokens, cap and a
// window of 4096, 848 MB in 134 us (6.3 TB/s); 4 sequences of 32k with slopes, 1.02 GB in
// 153 us (6.6 TB/s).  Beyond 8 columns per KV head the tiles' arithmetic takes over:
// FP8 pools, 48 sequences x 4 queries, 195 MB in 57 us (3.4 TB/s); 96 sequences x 3
// queries of 64 dims, 186 MB in 66 us (2.8 TB/s).
//
// Sequences cut by range boundaries leave partials, which a second kernel merges,
// a warp per output row.  (In plain decode the last warp to finish a KV head
// merges all its rows; with 32 columns per KV head and sequences cut over tens of
// ranges that took longer than the walk: 48 sequences x 4 queries over FP8 pools
// 79 us with it.)
#include "pa_launch.cuh"

#include <cmath>

#include "pa_decode_impl.h"

namespace pa {
namespace {

struct MergeParams {
  void* out;
  const int4* cuts;
  const float* part_ml;
  const float* part_o;
  int32_t* error_flag;
  int ranges;
  int rows;          // num_seqs * seq_rows
  int seq_rows;      // num_queries * num_heads
  float v_scale;
};

// WARPS warps per row: few rows, whose sequences are cut over many ranges, get all
// 8 of a CTA.  One / eight warps, whole call: 64 rows (2 sequences of 8k) 47.7 / 17.4 us,
// 1024 rows 38.6 / 36.7, 2048 rows 134.0 / 135.3, 6144 rows 56.7 / 66.7.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(256) pa_merge_kernel(const __grid_constant__ MergeParams p) {
  constexpr int DL = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WARPS;
  const int row = blockIdx.x * (8 / WARPS) + warp / WARPS;
  if (row >= p.rows) return;  // (all warps of a row alike)
  griddep_wait();
  griddep_launch_dependents();
  const int s = row / p.seq_rows, in_seq = row - s * p.seq_rows;
  const int4 cut = __ldcg(p.cuts + s);
  if (cut.w != kCutMerge) return;
  if (!cut_holds(cut.x, cut.y, cut.z, cut.w, p.ranges)) {
    if (lane == 0) report(p.error_flag, PA_DEVERR_STATE);
    return;
  }
  MergedRow<DL> m = merge_row<D>(p.part_ml, p.part_o, cut, p.seq_rows, in_seq, lane, part, WARPS);
  if constexpr (WARPS > 1) {
    __shared__ float parts[WARPS][DL + 2][32];
    parts[part][DL][lane] = m.m;
    parts[part][DL + 1][lane] = m.l;
#pragma unroll
    for (int i = 0; i < DL; ++i) parts[part][i][lane] = m.o[i];
    __syncthreads();
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) m.m = fmaxf(m.m, parts[w][DL][lane]);
    const float ref = m.m == -INFINITY ? 0.f : m.m;
    m.l = 0.f;
#pragma unroll
    for (int i = 0; i < DL; ++i) m.o[i] = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = ex2_ftz(parts[w][DL][lane] - ref);
      m.l = fmaf(f, parts[w][DL + 1][lane], m.l);
#pragma unroll
      for (int i = 0; i < DL; ++i) m.o[i] = fmaf(f, parts[w][i][lane], m.o[i]);
    }
  }
  const float inv = m.l > 0.f ? p.v_scale / m.l : 0.f;
  T* out = static_cast<T*>(p.out) + (size_t)row * D + lane * DL;
#pragma unroll
  for (int i = 0; i < DL; ++i) out[i] = T(m.o[i] * inv);
}

template <typename T, int D>
int launch_merge(const DecodeParams& prm, cudaStream_t stream) {
  MergeParams mp{prm.out, prm.cuts, prm.part_ml, prm.part_o, prm.error_flag, prm.num_ranges, 0,
                 prm.num_queries * prm.num_heads, prm.v_scale};
  mp.rows = prm.num_seqs * mp.seq_rows;
  const bool few = mp.rows <= 8 * prm.sm_count;
  const cudaError_t e =
      few ? launch_pdl(pa_merge_kernel<T, D, 8>, dim3(mp.rows), dim3(256), 0, stream, mp)
          : launch_pdl(pa_merge_kernel<T, D, 1>, dim3((mp.rows + 7) / 8), dim3(256), 0, stream, mp);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "launch pa_merge_kernel");
}

int launch_walk(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool f32,
                bool kv_fp8);

}  // namespace

int launch_mod(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool f32,
               bool kv_fp8) {
  const int rc = launch_walk(prm, pl, dev, stream, head_size, f32, kv_fp8);
  if (rc != PA_OK || pl.R == 1) return rc;  // one range cuts nothing
  if (f32) return head_size == 64 ? launch_merge<float, 64>(prm, stream) : launch_merge<float, 128>(prm, stream);
  return head_size == 64 ? launch_merge<__nv_bfloat16, 64>(prm, stream)
                         : launch_merge<__nv_bfloat16, 128>(prm, stream);
}

namespace {

int launch_walk(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool f32,
                bool kv_fp8) {
  const bool wide = prm.group * prm.num_queries > 8;  // two to four warps per KV head
  if (f32) {
    if (head_size == 64) {
      if (prm.group <= 2) return launch_typed<float, 64, 2, 0, false, kWalkMod>(prm, pl, dev, stream);
      return prm.group <= 4 ? launch_typed<float, 64, 4, 0, false, kWalkMod>(prm, pl, dev, stream)
                            : launch_typed<float, 64, 8, 0, false, kWalkMod>(prm, pl, dev, stream);
    }
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

extern "C" size_t pa_decode_mod_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                               int head_size, int kv_dtype, int num_ranges) {
  if (kv_dtype != PA_F32 && kv_dtype != PA_BF16 && kv_dtype != PA_FP8_E4M3) return 0;
  return pa::walk_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, num_ranges, num_queries,
                                 kv_dtype == PA_F32 ? 4 : kv_dtype == PA_BF16 ? 2 : 1);
}
