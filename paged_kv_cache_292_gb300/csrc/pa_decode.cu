// Host side of paged decode: the launch plan (heads per CTA, ranges, stage
// ring), the tensor maps of the pools, argument checks and the C entry
// points.  The kernel itself is in pa_decode_kernel.cuh.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "../../include/pagedattn.h"
#include "pa_decode_impl.h"
#include "pa_decode_kernel.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_plan.h"
#include "pa_schedule.h"

namespace pa {

EncodeTiledFn encode_tiled_fn() {
  static const EncodeTiledFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return static_cast<EncodeTiledFn>(nullptr);
    }
    return reinterpret_cast<EncodeTiledFn>(f);
  }();
  return fn;
}

// A tensor map that goes on where the memory ends is not safe even if every box lies in
// the pool: random multi-query calls over maps of 2^31 rows ended with an illegal
// address about once in 2000, with maps that end with the pools none of 86000 did.
uint64_t rows_of_pools(const void* k, const void* v, uint64_t row_bytes) {
  static const PFN_cuPointerGetAttributes_v7000 attributes_of = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuPointerGetAttributes", &f, 7000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      f = nullptr;
    }
    return reinterpret_cast<PFN_cuPointerGetAttributes_v7000>(f);
  }();
  uint64_t rows = 1ull << 31;
  for (const void* p : {k, v}) {
    CUdeviceptr start = 0;
    size_t size = 0;
    CUpointer_attribute what[2] = {CU_POINTER_ATTRIBUTE_RANGE_START_ADDR, CU_POINTER_ATTRIBUTE_RANGE_SIZE};
    void* out[2] = {&start, &size};
    const CUdeviceptr at = reinterpret_cast<CUdeviceptr>(p);
    const CUresult r = attributes_of == nullptr ? CUDA_ERROR_NOT_FOUND
                                                : in_context([&] { return attributes_of(2, what, out, at); });
    if (r != CUDA_SUCCESS) size = 0;
    const uint64_t mine = rows_behind(start, size, at, row_bytes);
    if (mine == 0) {
      fail(PA_ERR_INVALID_ARG, "pa_decode: the driver does not know the pools' memory; num_physical_blocks is needed");
      return 0;
    }
    if (mine < rows) rows = mine;
  }
  return rows;
}

namespace {

int validate(const void* out, const void* query, const void* k_cache, const void* v_cache,
             const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_heads,
             int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq, float scale,
             int dtype, int num_physical_blocks, int num_ranges) {
  if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens)
    return fail(PA_ERR_INVALID_ARG, "pa_decode: null tensor pointer");
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0)
    return fail(PA_ERR_INVALID_ARG, "pa_decode: sizes must be positive");
  if (num_heads % num_kv_heads != 0)
    return fail(PA_ERR_INVALID_ARG, "pa_decode: num_heads %d not a multiple of num_kv_heads %d",
                num_heads, num_kv_heads);
  if (num_heads / num_kv_heads > kMaxQueryGroup)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode: query group %d > %d", num_heads / num_kv_heads,
                kMaxQueryGroup);
  if (head_size != 64 && head_size != 128)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode: head_size %d (built: 64, 128)", head_size);
  if (block_size > 4096) return fail(PA_ERR_UNSUPPORTED, "pa_decode: block_size %d > 4096", block_size);
  if ((long long)max_blocks_per_seq * block_size > (1ll << 30))
    return fail(PA_ERR_INVALID_ARG, "pa_decode: max context %lld too large",
                (long long)max_blocks_per_seq * block_size);
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "pa_decode: dtype %d", dtype);
  if (!aligned(out, 16) || !aligned(query, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4))
    return fail(PA_ERR_INVALID_ARG, "pa_decode: tensors must be 16-byte aligned");
  if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "pa_decode: scale not finite");
  if (num_ranges > kMaxRanges)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode: num_ranges %d > %d", num_ranges, kMaxRanges);
  if (num_physical_blocks < 0 || num_ranges < 0)
    return fail(PA_ERR_INVALID_ARG, "pa_decode: negative num_physical_blocks or num_ranges");
  return PA_OK;
}

// The pools seen by the tensor copies: 4-D byte tensors (byte within a
// 128-byte chunk, chunk within a head group's row, head group, token row)
// with strides (1, 128, group row bytes, token row bytes).  A box is
// (128, lines, 1, box_rows); its lines past the group's row are outside the
// tensor, so they arrive zero-filled (requests to L2, but no reads of memory).
// Encoded for every call (about 0.1 us each): nothing is kept by a pool's address.
int make_tensor_maps(DecodeParams* prm, const Plan& pl, int num_kv_heads, int head_size, int kv_elt,
                     int block_size, int num_physical_blocks) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return fail(PA_ERR_CUDA, "pa_decode: the driver has no cuTensorMapEncodeTiled");
  const uint64_t token_bytes = (uint64_t)num_kv_heads * head_size * kv_elt;
  const uint64_t rows = num_physical_blocks > 0 ? (uint64_t)num_physical_blocks * block_size
                                                : rows_of_pools(prm->k_cache, prm->v_cache, token_bytes);
  if (rows == 0) return PA_ERR_INVALID_ARG;
  if (rows > (1ull << 31))
    return fail(PA_ERR_UNSUPPORTED, "pa_decode: %llu token rows in the pool (at most 2^31)",
                (unsigned long long)rows);
  const cuuint64_t dims[4] = {kLine, pl.row_bytes / kLine, (cuuint64_t)pl.HG, rows};
  const cuuint64_t strides[3] = {kLine, pl.row_bytes, token_bytes};
  const cuuint32_t box[4] = {kLine, pl.lines, 1u, pl.box_rows};
  const cuuint32_t estride[4] = {1u, 1u, 1u, 1u};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = in_context([&] {
      return enc(i ? &prm->tm_v : &prm->tm_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4,
                 const_cast<void*>(i ? prm->v_cache : prm->k_cache), dims, strides, box,
                 estride, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
    if (r != CUDA_SUCCESS)
      return fail(PA_ERR_CUDA, "pa_decode: cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  }
  return PA_OK;
}

template <typename T, int D>
int launch_dtype(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream,
                 bool kv_fp8 = false) {
  if constexpr (sizeof(T) == 2) {
    if (kv_fp8) {
      if (prm.num_queries == 1) return launch_typed<T, D, 8, 0, true>(prm, pl, dev, stream);
      return prm.group * prm.num_queries <= 8 ? launch_typed<T, D, 8, 1, true>(prm, pl, dev, stream)
                                               : launch_typed<T, D, 8, 2, true>(prm, pl, dev, stream);
    }
    if (prm.num_queries > 1)  // (query, head) columns in one or two 8-wide MMA tiles
      return prm.group * prm.num_queries <= 8 ? launch_typed<T, D, 8, 1>(prm, pl, dev, stream)
                                               : launch_typed<T, D, 8, 2>(prm, pl, dev, stream);
    return launch_typed<T, D, 8>(prm, pl, dev, stream);  // the MMA consumer pads G to 8
  } else {
    const int G = prm.group;
    if (G <= 1) return launch_typed<T, D, 1>(prm, pl, dev, stream);
    if (G <= 2) return launch_typed<T, D, 2>(prm, pl, dev, stream);
    if (G <= 4) return launch_typed<T, D, 4>(prm, pl, dev, stream);
    return launch_typed<T, D, 8>(prm, pl, dev, stream);
  }
}

}  // namespace

int decode_validate(const void* out, const void* query, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_queries,
                    int num_heads, int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq,
                    float scale, int dtype, int num_physical_blocks, int num_ranges) {
  int rc = validate(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_heads,
                    num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, dtype,
                    num_physical_blocks, num_ranges);
  if (rc != PA_OK) return rc;
  if (num_queries < 1) return fail(PA_ERR_INVALID_ARG, "pa_decode_mq: num_queries %d < 1", num_queries);
  if (num_queries > 1 && dtype != PA_BF16)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode_mq: several queries need bf16");
  if (num_queries > 1 && (num_heads / num_kv_heads) * num_queries > kMaxColumns)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode_mq: group size x queries = %d > %d",
                (num_heads / num_kv_heads) * num_queries, kMaxColumns);
  return PA_OK;
}

// fixed_scratch: when set and `workspace` is NULL, the scratch comes from this
// provider (given the plan's byte count, it returns a device buffer that keeps
// earlier contents, or an error) instead of the library's growable buffer;
// its merge tickets are then cleared on `stream` right before the launch,
// after every check has passed.
int decode_impl_q(void* out, const void* query, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                  int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                  int max_blocks_per_seq, float scale, void* stream, int dtype,
                  int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                  int32_t* error_flag, bool kv_fp8, float k_scale,
                  float v_scale, const void* k_new, const void* v_new,
                  ScratchProvider fixed_scratch, DecodeExtras* extras, const TokenScales* int8) {
  clear_error();
  if (k_new != nullptr || v_new != nullptr) {
    if (k_new == nullptr || v_new == nullptr)
      return fail(PA_ERR_INVALID_ARG, "pa_decode_append: k_new and v_new are both needed");
    if (dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "pa_decode_append: bf16 queries and pools only");
    if (!aligned(k_new, 16) || !aligned(v_new, 16))
      return fail(PA_ERR_INVALID_ARG, "pa_decode_append: k_new / v_new not 16-byte aligned");
  }
  if (kv_fp8) {
    if (dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "pa_decode_fp8: query/out must be bf16");
    if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f)
      return fail(PA_ERR_INVALID_ARG, "pa_decode_fp8: scales must be finite and positive");
  }
  int rc = decode_validate(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, dtype,
                           num_physical_blocks, num_ranges);
  if (rc != PA_OK) return rc;
  DeviceInfo dev{};
  rc = current_device_info(&dev);
  if (rc != PA_OK) return rc;
  const int elt = dtype == PA_F32 ? 4 : 2;
  Plan pl{};
  const PlanShape shape{num_heads, num_kv_heads, head_size, num_queries, kv_fp8 ? 1 : elt, elt, block_size, int8 != nullptr};
  rc = make_plan(shape, num_seqs, num_ranges, dev, extras != nullptr, &pl);
  if (rc != PA_OK) return rc;
  int32_t* counters = nullptr;
  ScratchHold hold;  // scratch of the library's own, until the launches are queued
  bool clear_tickets = workspace == nullptr && fixed_scratch != nullptr;
  size_t partials = 0;  // where they begin
  if (extras != nullptr) {
    if ((long long)num_seqs * num_queries * num_heads > 1 << 30)
      return fail(PA_ERR_UNSUPPORTED, "pa_decode: %d sequences of %d rows", num_seqs, num_queries * num_heads);
    const size_t need = walk_bytes(num_seqs, num_heads, num_kv_heads, head_size, pl.R, num_queries);
    // (The rest behind a shared prefix gets a part of that call's buffer.)
    if (extras->walk != kWalkRest && workspace != nullptr) partials = kTicketRoom;
    if (workspace == nullptr) {
      rc = hold.of_stream(need, stream, &workspace);
      if (rc != PA_OK) return rc;
    } else if (workspace_bytes < partials + need) {
      return fail(PA_ERR_WORKSPACE, "pa_decode: workspace of %zu bytes, %zu needed", workspace_bytes, partials + need);
    } else if (!aligned(workspace, 256)) {
      return fail(PA_ERR_INVALID_ARG, "pa_decode: workspace not 256-byte aligned");
    }
  } else if (clear_tickets) {
    rc = fixed_scratch(pl.ws_total, &workspace);
    if (rc != PA_OK) return rc;
    workspace_bytes = pl.ws_total;
  }
  if (extras != nullptr) {
  } else if (workspace == nullptr && int8 != nullptr) {
    rc = hold.of_stream(pl.ws_partials, stream, &workspace, pl.ws_tickets, &counters);
    if (rc != PA_OK) return rc;
  } else if (workspace == nullptr) {
    rc = hold.plain(pl.ws_partials, pl.ws_tickets, stream, &workspace, &counters);
    if (rc != PA_OK) return rc;
  } else {
    if (workspace_bytes < pl.ws_total)
      return fail(PA_ERR_WORKSPACE, "pa_decode: workspace of %zu bytes, %zu needed", workspace_bytes,
                  pl.ws_total);
    if (!aligned(workspace, 256)) return fail(PA_ERR_INVALID_ARG, "pa_decode: workspace not 256-byte aligned");
    counters = reinterpret_cast<int32_t*>(static_cast<unsigned char*>(workspace) + pl.ws_late);
    if (pl.ws_late != 0) clear_tickets = true;
    partials = kTicketRoom;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace) + partials;
  DecodeParams prm{};
  prm.out = out;
  prm.q = query;
  prm.k_cache = k_cache;
  prm.v_cache = v_cache;
  prm.block_tables = block_tables;
  prm.context_lens = context_lens;
  prm.counters = counters;
  prm.part_ml = reinterpret_cast<float*>(ws + pl.ws_ml);
  prm.part_o = reinterpret_cast<float*>(ws + pl.ws_o);
  prm.error_flag = error_flag;
  prm.num_seqs = num_seqs;
  prm.num_heads = num_heads;
  prm.num_kv_heads = num_kv_heads;
  prm.group = num_heads / num_kv_heads;
  prm.block_size = block_size;
  prm.max_blocks_per_seq = max_blocks_per_seq;
  prm.heads_per_cta = pl.Hg;
  prm.num_head_groups = pl.HG;
  prm.num_ranges = pl.R;
  prm.num_physical_blocks = num_physical_blocks;
  prm.stages = pl.stages;
  prm.num_queries = num_queries;
  prm.split = pl.split;
  prm.q_slots = pl.q_slots;
  prm.row_bytes = pl.row_bytes;
  prm.pitch = pl.pitch;
  prm.q_bytes = pl.q_bytes;
  prm.stage_bytes = pl.stage_bytes;
  prm.lines = pl.lines;
  prm.box_rows = pl.box_rows;
  prm.box_bytes = pl.box_bytes;
  if (dtype == PA_BF16) {
    rc = make_tensor_maps(&prm, pl, num_kv_heads, head_size, kv_fp8 ? 1 : 2, block_size,
                          num_physical_blocks);
    if (rc != PA_OK) return rc;
  }
  prm.scale_log2 = (float)((double)scale * (double)k_scale * 1.4426950408889634);
  prm.v_scale = v_scale;
  prm.k_scale = k_scale;
  prm.k_new = k_new;
  prm.v_new = v_new;
  if (int8 != nullptr) {
    prm.k_scales = int8->k;
    prm.v_scales = int8->v;
  }
  if (extras != nullptr) {
    prm.sm_count = dev.sm_count;
    prm.cuts = reinterpret_cast<int4*>(ws + pl.ws_partials);
    extras->ranges = pl.R;
    extras->cuts = prm.cuts;
    extras->part_ml = prm.part_ml;
    extras->part_o = prm.part_o;
  }
  prm.window = kNoWindow;
  if (extras != nullptr && extras->walk == kWalkMod) {
    const double log2e = 1.4426950408889634;
    const double per_cap = extras->softcap > 0.f ? (double)scale * k_scale / extras->softcap : 0.0;
    // The tensor-core consumers take tanh from a power of two, fp32 calls tanhf.
    // Caps at the ends of fp32's range keep finite factors: any score reaches the
    // smallest caps, none gets near the largest.
    const double cap_in = dtype == PA_F32 ? per_cap : 2.0 * log2e * per_cap, most = FLT_MAX;
    prm.cap_in = (float)(cap_in > most ? most : cap_in < -most ? -most : cap_in);
    const double cap_out = extras->softcap * log2e;
    prm.cap_out = (float)(cap_out > most ? most : cap_out);
    prm.slopes = extras->alibi_slopes;
    prm.first_tokens = extras->first_tokens;
    prm.prefix_lens = extras->prefix_lens;
    if (extras->window > 0 && extras->window < kNoWindow) prm.window = extras->window;
  } else if (extras != nullptr) {
    prm.prefix_tokens = extras->prefix_tokens;
    prm.beside = extras->prefix_units > 0.f;
    prm.prefix_units = extras->prefix_units;
    prm.rest_ml = extras->rest_ml;
    prm.rest_o = extras->rest_o;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (clear_tickets) {
    const cudaError_t e = cudaMemsetAsync(counters, 0, pl.ws_tickets, st);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync(merge tickets)");
  }
  if (extras != nullptr && extras->walk == kWalkRest) {
    rc = extras->before(extras, extras->context);
    if (rc != PA_OK) return rc;
    prm.stall_tile = extras->stall_tile;
    prm.wait_limit_ns = extras->wait_limit_ns;
  } else {
    take_wait_test(&prm.stall_tile, &prm.wait_limit_ns);
  }
  if (k_new != nullptr && pl.split >= 2) {
    // Several consumer warps per KV head: the rows are written by their own
    // kernel, chained ahead of the decode, which then only reads them.
    rc = append_rows_impl(k_new, v_new, block_tables, context_lens, const_cast<void*>(k_cache),
                          const_cast<void*>(v_cache), num_seqs, num_queries, num_kv_heads, head_size,
                          block_size, max_blocks_per_seq, num_physical_blocks, stream, error_flag,
                          kv_fp8, k_scale, v_scale);
    if (rc != PA_OK) return rc;
    prm.k_new = prm.v_new = nullptr;
  }
  if (extras != nullptr)
    return extras->walk == kWalkMod ? launch_mod(prm, pl, dev.device, st, head_size, dtype == PA_F32, kv_fp8)
                                    : launch_rest(prm, pl, dev.device, st, head_size, kv_fp8);
  if (int8 != nullptr) return launch_int8(prm, pl, dev.device, st, head_size);
  if (dtype == PA_BF16) {
    return head_size == 64 ? launch_dtype<__nv_bfloat16, 64>(prm, pl, dev.device, st, kv_fp8)
                           : launch_dtype<__nv_bfloat16, 128>(prm, pl, dev.device, st, kv_fp8);
  }
  return head_size == 64 ? launch_dtype<float, 64>(prm, pl, dev.device, st)
                         : launch_dtype<float, 128>(prm, pl, dev.device, st);
}

int decode_impl(void* out, const void* query, const void* k_cache, const void* v_cache,
                const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                int num_heads, int num_kv_heads, int head_size, int block_size,
                int max_blocks_per_seq, float scale, void* stream, int dtype,
                int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                int32_t* error_flag) {
  return decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, 1,
                       num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                       stream, dtype, num_physical_blocks, workspace, workspace_bytes, num_ranges,
                       error_flag);
}

size_t decode_workspace_size_q(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                               int num_ranges, int num_queries) {
  if (num_queries < 1) return 0;
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 || num_ranges < 0 ||
      num_heads % num_kv_heads != 0)
    return 0;
  int R = num_ranges;
  if (R == 0) {
    DeviceInfo dev{};
    if (current_device_info(&dev) != PA_OK) return 0;
    // The head grouping depends on the element size; size for bf16, whose
    // larger groups leave more ranges per head group.
    const int split = column_split(num_heads / num_kv_heads, num_queries);
    R = default_ranges(dev, num_kv_heads / heads_per_cta(num_kv_heads, head_size, 2, kMaxGroupHeads / split));
  }
  return workspace_layout(num_seqs, num_heads, num_kv_heads, head_size, R, nullptr, num_queries);
}

size_t walk_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size, int num_ranges,
                           int num_queries, int elt, bool any_block) {
  if (num_queries < 1 || num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_size <= 0 ||
      num_ranges < 0 || num_heads % num_kv_heads != 0)
    return 0;
  if (num_ranges > 0) return walk_bytes(num_seqs, num_heads, num_kv_heads, head_size, num_ranges, num_queries);
  DeviceInfo dev{};
  if (current_device_info(&dev) != PA_OK) return 0;
  const PlanShape shape{num_heads, num_kv_heads, head_size, num_queries, elt, elt == 4 ? 4 : 2, kTile};
  const size_t need = walk_workspace(shape, num_seqs, dev, any_block);
  clear_error();  // (plans of other block sizes)
  return need;
}

size_t decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                             int num_ranges) {
  return decode_workspace_size_q(num_seqs, num_heads, num_kv_heads, head_size, num_ranges, 1);
}

}  // namespace pa

extern "C" int pa_decode(void* out, const void* query, const void* k_cache, const void* v_cache,
                         const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                         int num_heads, int num_kv_heads, int head_size, int block_size,
                         int max_blocks_per_seq, float scale, void* stream, int dtype) {
  return pa::decode_impl(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                         num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                         stream, dtype, 0, nullptr, 0, 0, nullptr);
}

extern "C" int pa_decode_ws(void* out, const void* query, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens,
                            int num_seqs, int num_heads, int num_kv_heads, int head_size,
                            int block_size, int max_blocks_per_seq, float scale, void* stream,
                            int dtype, void* workspace, size_t workspace_bytes) {
  if (workspace == nullptr) {
    pa::clear_error();
    return pa::fail(PA_ERR_INVALID_ARG, "pa_decode_ws: null workspace");
  }
  return pa::decode_impl(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                         num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                         stream, dtype, 0, workspace, workspace_bytes, 0, nullptr);
}

extern "C" int pa_decode_ex(void* out, const void* query, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens,
                            int num_seqs, int num_heads, int num_kv_heads, int head_size,
                            int block_size, int max_blocks_per_seq, float scale, void* stream,
                            int dtype, int num_physical_blocks, void* workspace,
                            size_t workspace_bytes, int num_ranges, int32_t* error_flag) {
  return pa::decode_impl(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                         num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                         stream, dtype, num_physical_blocks, workspace, workspace_bytes, num_ranges,
                         error_flag);
}

extern "C" int pa_decode_append(void* out, const void* query, const void* k_new, const void* v_new,
                                void* k_cache, void* v_cache, const int32_t* block_tables,
                                const int32_t* context_lens, int num_seqs, int num_heads,
                                int num_kv_heads, int head_size, int block_size,
                                int max_blocks_per_seq, float scale, void* stream, int dtype,
                                int num_physical_blocks, void* workspace, size_t workspace_bytes,
                                int num_ranges, int32_t* error_flag) {
  if (k_new == nullptr || v_new == nullptr) {
    pa::clear_error();
    return pa::fail(PA_ERR_INVALID_ARG, "pa_decode_append: null k_new / v_new");
  }
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, 1,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                           stream, dtype, num_physical_blocks, workspace, workspace_bytes, num_ranges,
                           error_flag, false, 1.f, 1.f, k_new, v_new);
}

extern "C" int pa_decode_fp8_append(void* out, const void* query, const void* k_new, const void* v_new,
                                    void* k_cache, void* v_cache, const int32_t* block_tables,
                                    const int32_t* context_lens, int num_seqs, int num_heads,
                                    int num_kv_heads, int head_size, int block_size,
                                    int max_blocks_per_seq, float scale, float k_scale, float v_scale,
                                    void* stream, int num_physical_blocks, void* workspace,
                                    size_t workspace_bytes, int num_ranges, int32_t* error_flag) {
  if (k_new == nullptr || v_new == nullptr) {
    pa::clear_error();
    return pa::fail(PA_ERR_INVALID_ARG, "pa_decode_fp8_append: null k_new / v_new");
  }
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, 1,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                           stream, PA_BF16, num_physical_blocks, workspace, workspace_bytes, num_ranges,
                           error_flag, true, k_scale, v_scale, k_new, v_new);
}

extern "C" size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                           int head_size, int num_ranges) {
  return pa::decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, num_ranges);
}

extern "C" int pa_decode_mq(void* out, const void* query, const void* k_cache, const void* v_cache,
                            const int32_t* block_tables, const int32_t* context_lens,
                            int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                            int head_size, int block_size, int max_blocks_per_seq, float scale,
                            void* stream, int dtype, int num_physical_blocks, void* workspace,
                            size_t workspace_bytes, int num_ranges, int32_t* error_flag) {
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                           num_queries, num_heads, num_kv_heads, head_size, block_size,
                           max_blocks_per_seq, scale, stream, dtype, num_physical_blocks, workspace,
                           workspace_bytes, num_ranges, error_flag);
}

extern "C" int pa_decode_mq_append(void* out, const void* query, const void* k_new, const void* v_new,
                                   void* k_cache, void* v_cache, const int32_t* block_tables,
                                   const int32_t* context_lens, int num_seqs, int num_queries,
                                   int num_heads, int num_kv_heads, int head_size, int block_size,
                                   int max_blocks_per_seq, float scale, void* stream, int dtype,
                                   int num_physical_blocks, void* workspace, size_t workspace_bytes,
                                   int num_ranges, int32_t* error_flag) {
  if (k_new == nullptr || v_new == nullptr) {
    pa::clear_error();
    return pa::fail(PA_ERR_INVALID_ARG, "pa_decode_mq_append: null k_new / v_new");
  }
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                           num_queries, num_heads, num_kv_heads, head_size, block_size,
                           max_blocks_per_seq, scale, stream, dtype, num_physical_blocks, workspace,
                           workspace_bytes, num_ranges, error_flag, false, 1.f, 1.f, k_new, v_new);
}

extern "C" size_t pa_decode_mq_workspace_size(int num_seqs, int num_queries, int num_heads,
                                              int num_kv_heads, int head_size, int num_ranges) {
  return pa::decode_workspace_size_q(num_seqs, num_heads, num_kv_heads, head_size, num_ranges,
                                     num_queries);
}

extern "C" int pa_decode_fp8(void* out, const void* query, const void* k_cache, const void* v_cache,
                             const int32_t* block_tables, const int32_t* context_lens,
                             int num_seqs, int num_heads, int num_kv_heads, int head_size,
                             int block_size, int max_blocks_per_seq, float scale, float k_scale,
                             float v_scale, void* stream, int num_physical_blocks, void* workspace,
                             size_t workspace_bytes, int num_ranges, int32_t* error_flag) {
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, 1,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale,
                           stream, PA_BF16, num_physical_blocks, workspace, workspace_bytes,
                           num_ranges, error_flag, true, k_scale, v_scale);
}

extern "C" int pa_decode_fp8_mq(void* out, const void* query, const void* k_cache, const void* v_cache,
                                const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                                int num_queries, int num_heads, int num_kv_heads, int head_size,
                                int block_size, int max_blocks_per_seq, float scale, float k_scale,
                                float v_scale, void* stream, int num_physical_blocks, void* workspace,
                                size_t workspace_bytes, int num_ranges, int32_t* error_flag) {
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                           num_queries, num_heads, num_kv_heads, head_size, block_size,
                           max_blocks_per_seq, scale, stream, PA_BF16, num_physical_blocks, workspace,
                           workspace_bytes, num_ranges, error_flag, true, k_scale, v_scale);
}

extern "C" int pa_decode_fp8_mq_append(void* out, const void* query, const void* k_new, const void* v_new,
                                       void* k_cache, void* v_cache, const int32_t* block_tables,
                                       const int32_t* context_lens, int num_seqs, int num_queries,
                                       int num_heads, int num_kv_heads, int head_size, int block_size,
                                       int max_blocks_per_seq, float scale, float k_scale, float v_scale,
                                       void* stream, int num_physical_blocks, void* workspace,
                                       size_t workspace_bytes, int num_ranges, int32_t* error_flag) {
  if (k_new == nullptr || v_new == nullptr) {
    pa::clear_error();
    return pa::fail(PA_ERR_INVALID_ARG, "pa_decode_fp8_mq_append: null k_new / v_new");
  }
  return pa::decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs,
                           num_queries, num_heads, num_kv_heads, head_size, block_size,
                           max_blocks_per_seq, scale, stream, PA_BF16, num_physical_blocks, workspace,
                           workspace_bytes, num_ranges, error_flag, true, k_scale, v_scale, k_new, v_new);
}
