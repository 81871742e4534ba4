// The general decode call behind the C entry points of several translation units.
#pragma once

#include <vector_types.h>

#include "pa_internal.h"

namespace pa {

// What a call asks of the decode kernel beyond the plain step.
struct DecodeExtras {
  int walk;  // kWalkMod or kWalkRest
  // kWalkMod: modified scores
  float softcap = 0.f;
  const float* alibi_slopes = nullptr;
  int window = 0;
  const int32_t* first_tokens = nullptr;
  const int32_t* prefix_lens = nullptr;
  // kWalkRest: the tokens behind a shared prefix, left as (m, l, O) rows
  int prefix_tokens = 0;
  float prefix_units = 0.f;  // work of the prefix kernel launched just before (0: none)
  float* rest_ml = nullptr;
  float* rest_o = nullptr;
  // kWalkRest: queues what goes before the walk, once nothing but a launch can fail
  // any more, and sets the walk's settings of pa_test_stall_copy.
  int (*before)(DecodeExtras* self, void* context) = nullptr;
  void* context = nullptr;
  long long stall_tile = -1;
  unsigned long long wait_limit_ns = 0;
  // Set by the call, inside its scratch: how sequences were cut, and the partials.
  int ranges = 0;
  int4* cuts = nullptr;
  const float* part_ml = nullptr;
  const float* part_o = nullptr;
};

// Scratch of a call with extras (num_ranges 0: the default; elt: bytes of a pool
// element; any_block: not only for blocks that are multiples of 8).  0 for invalid sizes.
size_t walk_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_size, int num_ranges,
                           int num_queries, int elt, bool any_block = true);

// The argument checks every decode call makes.
int decode_validate(const void* out, const void* query, const void* k_cache, const void* v_cache,
                    const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_queries,
                    int num_heads, int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq,
                    float scale, int dtype, int num_physical_blocks, int num_ranges = 0);

int decode_impl_q(void* out, const void* query, const void* k_cache, const void* v_cache,
                  const int32_t* block_tables, const int32_t* context_lens, int num_seqs,
                  int num_queries, int num_heads, int num_kv_heads, int head_size, int block_size,
                  int max_blocks_per_seq, float scale, void* stream, int dtype,
                  int num_physical_blocks, void* workspace, size_t workspace_bytes, int num_ranges,
                  int32_t* error_flag, bool kv_fp8 = false, float k_scale = 1.f,
                  float v_scale = 1.f, const void* k_new = nullptr, const void* v_new = nullptr,
                  ScratchProvider fixed_scratch = nullptr, DecodeExtras* extras = nullptr);

}  // namespace pa
