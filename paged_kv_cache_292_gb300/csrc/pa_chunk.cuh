// Chunk attention's parts that its kernels share: a call's arguments, the walk of a
// CTA over its range of the list (pa_chunk_work.h), and the join of what range
// boundaries cut.
#pragma once

#include "../../include/pa_int8_cache.h"
#include "pa_chunk_work.h"
#include "pa_launch.cuh"

namespace pa {

// A call of any of the entry points.
struct ChunkCall {
  void* out;
  const void* query;
  const void* k_cache;
  const void* v_cache;
  const float* k_scales;  // int8
  const float* v_scales;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* seq_starts;
  int num_tokens;
  int num_queries;  // > 0: tokens of every sequence, instead of seq_starts and num_tokens
  int num_seqs, num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq;
  float scale;
  void* stream;
  int dtype;
  bool int8;
  int num_physical_blocks;
  void* workspace;
  size_t workspace_bytes;
  int32_t* error_flag;

  long long tokens() const { return num_queries > 0 ? (long long)num_seqs * num_queries : num_tokens; }
};

// The argument checks, and the call itself.
int prefill_validate(const ChunkCall& c);
int prefill_impl(const ChunkCall& c);

struct ChunkParams {
  CUtensorMap tm_q;        // (element, head, token)
  CUtensorMap tm_k, tm_v;  // (element of a panel, row of 8, panel, group of 8 token rows, KV head); int8: (D, KV head, token row)
  const void* q;
  void* out;
  const void* k_cache;
  const void* v_cache;
  const float* k_scales;  // [block][KV head][row of the block]
  const float* v_scales;
  const int32_t* tables;
  const int32_t* context_lens;
  const int32_t* seq_starts;  // nullptr: num_queries tokens each
  int32_t* error_flag;
  float* part_ml;  // [2 * CTAs][256][2]
  float* part_o;   // [2 * CTAs][2][D / 4][128][4]: a thread's row side by side with its neighbours'
  // [CTAs][2]: the item in which a CTA's range begins, (sequence, head, pair, first tile), and its
  // (first row of the token buffer, tokens, 0, 0).
  int4* cuts;
  int num_tokens, num_seqs, num_queries, num_heads, kv_heads, group, tile_tokens, item_units;
  int block_size, max_blocks, max_tokens, num_physical_blocks, box_rows;
  // Scores are scale_log2 * sign * <q, k> with scale_log2 > 0, so that the largest product
  // (times sign) is the largest score; fp32: scale_log2 has the sign.
  float scale_log2, sign;
  unsigned long long wait_limit_ns;
  long long stall_tile;  // tests of the bounded waits: tile of every CTA whose copies are withheld (-1: none)
};

// fp32 pools (pa_prefill_f32.cu): queues both launches.
int launch_chunks_f32(const ChunkParams& prm, const DeviceInfo& dev, cudaStream_t stream, int head_size);

// (what follows has internal linkage: every translation unit has its own copy)
namespace {

// A sequence's rows and lengths, inside the buffers whatever the arrays hold.
struct ChunkRow {
  int row0, n, ctx;
};
__device__ __forceinline__ ChunkRow chunk_row(const ChunkParams& p, int s, bool report_it) {
  ChunkRow r;
  if (p.seq_starts == nullptr) {
    r.row0 = s * p.num_queries;
    r.n = p.num_queries;
  } else {
    const int a = __ldg(p.seq_starts + s), b = __ldg(p.seq_starts + s + 1);
    r.row0 = min(max(a, 0), p.num_tokens);
    const int end = min(max(b, 0), p.num_tokens);
    r.n = max(end - r.row0, 0);
    if (report_it && (a != r.row0 || b != end || b < a)) report(p.error_flag, PA_DEVERR_CONTEXT_LEN);
  }
  const int c = __ldg(p.context_lens + s);
  r.ctx = min(max(c, 0), p.max_tokens);
  if (report_it && c != r.ctx) report(p.error_flag, PA_DEVERR_CONTEXT_LEN);
  return r;
}

// The items of a CTA's range, one after another; every role walks them.
struct ChunkItems {
  int64_t ua, ub, start;  // the range, and the item's first unit
  int seq, head, pair;
  ChunkRow row;
  ChunkSeq cs;
  int t0, t1, tiles;
  int item_units;

  __device__ __forceinline__ void load(const ChunkParams& p) {
    row = chunk_row(p, seq, false);
    cs = ChunkSeq{row.n, row.ctx - row.n, p.tile_tokens, item_units};
  }
  __device__ __forceinline__ void set() {
    tiles = cs.tiles(pair);
    t0 = chunk_tile_at(ua - start, tiles, cs.item);
    t1 = chunk_tile_at(ub - start, tiles, cs.item);
  }
  // False behind the range's last item.
  __device__ __forceinline__ bool next(const ChunkParams& p) {
    start += cs.item + tiles;
    if (start >= ub) return false;
    if (++pair == cs.pairs()) {
      pair = 0;
      if (++head == p.kv_heads) {
        head = 0;
        do {
          if (++seq >= p.num_seqs) return false;
          load(p);
        } while (row.n == 0);
      }
    }
    set();
    return true;
  }
  __device__ __forceinline__ bool two() const { return cs.two(pair); }
};

// This CTA's range of the list and the item that it begins in, found by all of its threads
// (`shared`: kThreads / 32 + 8 long long).  False: no range for it.
template <int kThreads>
__device__ __forceinline__ bool chunk_begin(const ChunkParams& p, ChunkItems* at, long long* shared) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  // The sequence, its first unit and its units per head; (first row, tokens, context); pair, its first unit.
  long long* found = shared + kWarps;
  int* found_row = reinterpret_cast<int*>(found + 5);
  const bool one_each = p.num_seqs <= kThreads;  // a thread has one sequence at most
  ChunkRow row{0, 0, 0};
  int64_t units = 0, before = 0;  // of the thread's sequence, per head; of the sequences before it
  at->item_units = p.item_units;
  // The units of sequences base .. base + kThreads - 1, and each thread's place among them.
  auto scan = [&](int base, bool report_it) -> int64_t {
    units = 0;
    if (base + tid < p.num_seqs) {
      row = chunk_row(p, base + tid, report_it);
      units = ChunkSeq{row.n, row.ctx - row.n, p.tile_tokens, at->item_units}.units();
    }
    const int64_t mine = units * p.kv_heads, incl = warp_incl_scan_ll(mine, lane);
    __syncthreads();
    if (lane == 31) shared[warp] = incl;
    __syncthreads();
    int64_t all = 0;
    before = incl - mine;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const int64_t w = shared[i];
      if (i < warp) before += w;
      all += w;
    }
    return all;
  };
  if (tid < 5) found[tid] = -1;
  int64_t total = 0;
  for (int b = 0; b < p.num_seqs; b += kThreads) total += scan(b, cta == 0);
  // A list that leaves CTAs without a range is cut finer: there, an item's costs are paid side by
  // side.  (16 tokens on 1k: 23.6 -> 19.3 us; batches that fill the SMs take 2 to 20% longer so.  fp32, whose
  // tiles take longest: 3 prompts of up to 200 tokens 44 -> 32; bf16 with nothing for an item, 19 -> 23.)
  if (at->item_units > 0 && chunk_ranges(total, gridDim.x, at->item_units) < (int)gridDim.x) {
    at->item_units = at->item_units > 1 ? 1 : 0;
    total = 0;
    for (int b = 0; b < p.num_seqs; b += kThreads) total += scan(b, false);
  }
  const int ranges = chunk_ranges(total, gridDim.x, at->item_units);
  bool here = total > 0 && cta < ranges;
  if (here) {
    at->ua = range_start(cta, total, ranges);
    at->ub = range_start(cta + 1, total, ranges);
    int64_t earlier = 0;
    for (int b = 0; b < p.num_seqs; b += kThreads) {
      const int64_t all = one_each ? total : scan(b, false);
      const int64_t first = earlier + before;
      if (units > 0 && first <= at->ua && at->ua < first + units * p.kv_heads) {
        found[0] = b + tid;
        found[1] = first;
        found[2] = units;
        found_row[0] = row.row0;
        found_row[1] = row.n;
        found_row[2] = row.ctx;
      }
      earlier += all;
    }
    __syncthreads();
    at->seq = (int)found[0];
    here = at->seq >= 0;
  }
  if (here) {
    at->row = ChunkRow{found_row[0], found_row[1], found_row[2]};
    at->cs = ChunkSeq{at->row.n, at->row.ctx - at->row.n, p.tile_tokens, at->item_units};
    const int64_t per_head = found[2], in_seq = at->ua - found[1];
    at->head = ((in_seq | per_head) >> 32) == 0 ? (int)((uint32_t)in_seq / (uint32_t)per_head) : (int)(in_seq / per_head);
    const int64_t in_head = in_seq - at->head * per_head;
    for (int j = tid; j < at->cs.pairs(); j += kThreads) {
      const int64_t a = at->cs.before(j);
      if (a <= in_head && in_head < a + at->cs.item_units(j)) {
        found[3] = j;
        found[4] = a;
      }
    }
    __syncthreads();
    at->pair = (int)found[3];
    at->start = at->ua - in_head + found[4];
    at->set();
    here = at->pair >= 0;
  }
  if (tid == 0) {
    int4 item = make_int4(-1, 0, 0, 0), rows = make_int4(0, 0, 0, 0);
    if (here) {
      const int first = at->pair * 2 * p.tile_tokens;
      item = make_int4(at->seq, at->head, at->pair, at->t0 < at->tiles ? at->t0 : 0);
      rows = make_int4(at->row.row0 + first, min(at->row.n - first, 2 * p.tile_tokens), 0, 0);
    }
    p.cuts[2 * cta] = item;
    p.cuts[2 * cta + 1] = rows;
  }
  return here;
}

// ---------------------------------------------------------------------------
// Join: the rows of the items that range boundaries cut, by log-sum-exp.  kJoinBlocks blocks
// belong to every boundary, and those of an item's boundaries share its rows.  With many rows
// a block (and few parts: the list is long, then) a warp takes 32 of them, a lane each, and a slice of
// the dims, so that its loads lie side by side; with few (and perhaps many parts) eight warps share
// a row, and a lane has four dims.  (16 tokens on 4k, 17 parts: 43 us with the first boundary's
// blocks alone, 29 with all.)
// ---------------------------------------------------------------------------
constexpr int kJoinBlocks = 4, kSlice = 32;  // dims of a warp where there are many rows

template <typename T, int D>
__global__ void __launch_bounds__(256, 4) pa_prefill_join(const __grid_constant__ ChunkParams p) {
  constexpr int kLanes = D / 4;  // lanes that hold four dims (the others repeat them)
  const int lane = threadIdx.x & 31, dims = lane % kLanes, warp = threadIdx.x >> 5;
  const int b = blockIdx.x + 1, ctas = gridDim.x + 1;
  griddep_wait();
  griddep_launch_dependents();
  const int4 cut = __ldcg(p.cuts + 2 * b), before = __ldcg(p.cuts + 2 * b - 2), item = __ldcg(p.cuts + 2 * b + 1);
  if (cut.x < 0 || cut.w == 0) return;  // no such range, or it begins with an item
  auto same = [&](const int4& o) { return o.x == cut.x && o.y == cut.y && o.z == cut.z && o.w != 0; };
  // The CTAs whose ranges begin in the item are first .. first + parts - 2.
  int first = b, parts = 2;
  if (same(before)) {
    for (int i = b - 1;; i -= 32) {
      const unsigned run = __ballot_sync(0xffffffffu, i - lane >= 1 && same(__ldcg(p.cuts + 2 * max(i - lane, 1))));
      first -= __ffs(~run) == 0 ? 32 : __ffs(~run) - 1;
      if (run != 0xffffffffu) break;
    }
  }
  for (int i = b + 1;; i += 32) {
    const bool more = i + lane < ctas && same(__ldcg(p.cuts + 2 * min(i + lane, ctas - 1)));
    const unsigned run = __ballot_sync(0xffffffffu, more);
    parts += __ffs(~run) == 0 ? 32 : __ffs(~run) - 1;
    if (run != 0xffffffffu) break;
  }
  parts += b - first;
  const int blocks = (parts - 1) * kJoinBlocks, block = (b - first) * kJoinBlocks + blockIdx.y;
  // (After a timeout of the kernel before the list may hold anything: stay inside.)
  const int tokens = item.y;
  if (cut.y < 0 || cut.y >= p.kv_heads || item.x < 0 || tokens < 0 || tokens > 2 * p.tile_tokens ||
      item.x + tokens > p.num_tokens) {
    if (threadIdx.x == 0) report(p.error_flag, PA_DEVERR_STATE);
    return;
  }
  const int rows = tokens * p.group;
  // Part k: CTA first - 1 + k, the first in its second slot, the others in their first.
  auto slot = [&](int k) -> size_t { return (size_t)2 * (first - 1 + k) + (k == 0 ? 1 : 0); };
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  const float4* po = reinterpret_cast<const float4*>(p.part_o);
  if (rows > 8 * blocks) {
    constexpr int kSlices = D / kSlice;
    for (int i = block * 8 + warp; i < 2 * (kChunkRows / 32) * kSlices; i += 8 * blocks) {
      const int d0 = (i % kSlices) * kSlice, r = (i / kSlices) * 32 + lane, tile = r / kChunkRows, in_tile = r % kChunkRows;
      const int t = in_tile / p.group, tok = tile * p.tile_tokens + t;
      const bool real = t < p.tile_tokens && tok < tokens;
      if (!__any_sync(0xffffffffu, real)) continue;
      float m = -INFINITY, l = 0.f, acc[kSlice];
#pragma unroll
      for (int e = 0; e < kSlice; ++e) acc[e] = 0.f;
      if (!real) continue;  // (nothing below is for the whole warp)
      for (int k = 0; k < parts; ++k) {
        const float2 a = __ldcg(ml + slot(k) * (2 * kChunkRows) + r);
        float4 o[kSlice / 4];
#pragma unroll
        for (int e = 0; e < kSlice / 4; ++e)
          o[e] = __ldcg(po + ((slot(k) * 2 + tile) * (D / 4) + d0 / 4 + e) * kChunkRows + in_tile);
        if (a.y == 0.f) continue;  // no token seen: O may be anything
        const float mn = fmaxf(m, a.x), keep = ex2_ftz(m - mn), f = ex2_ftz(a.x - mn);
        m = mn;
        l = fmaf(l, keep, f * a.y);
#pragma unroll
        for (int e = 0; e < kSlice / 4; ++e) {
          acc[4 * e] = fmaf(acc[4 * e], keep, f * o[e].x);
          acc[4 * e + 1] = fmaf(acc[4 * e + 1], keep, f * o[e].y);
          acc[4 * e + 2] = fmaf(acc[4 * e + 2], keep, f * o[e].z);
          acc[4 * e + 3] = fmaf(acc[4 * e + 3], keep, f * o[e].w);
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < kSlice; ++e) acc[e] *= inv;
      T* out = static_cast<T*>(p.out) +
               ((size_t)(item.x + tok) * p.num_heads + cut.y * p.group + (in_tile - t * p.group)) * D + d0;
#pragma unroll
      for (int e = 0; e < kSlice; e += 16 / (int)sizeof(T)) {
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(out + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        else
          *reinterpret_cast<uint4*>(out + e) =
              make_uint4(pack_bf16x2(acc[e], acc[e + 1]), pack_bf16x2(acc[e + 2], acc[e + 3]),
                         pack_bf16x2(acc[e + 4], acc[e + 5]), pack_bf16x2(acc[e + 6], acc[e + 7]));
      }
    }
    return;
  }
  __shared__ float shared_parts[8][6][32];
  for (int i = block; i < rows; i += blocks) {
    const int tok = i / p.group, g = i - tok * p.group;
    const int tile = tok >= p.tile_tokens ? 1 : 0;
    const int in_tile = (tok - tile * p.tile_tokens) * p.group + g;
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int k0 = warp; k0 < parts; k0 += 32 * 8) {
      const int k = k0 + lane * 8, here = min(32, (parts - k0 + 7) / 8);
      float2 a = make_float2(-INFINITY, 0.f);
      if (k < parts) a = __ldcg(ml + slot(k) * (2 * kChunkRows) + tile * kChunkRows + in_tile);
      if (a.y == 0.f) a.x = -INFINITY;  // no token seen: no weight
      float top = a.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
      const float keep = ex2_ftz(m - ref);
      const float wa = a.y == 0.f ? 0.f : ex2_ftz(a.x - ref);
      m = mn;
      float lw = wa * a.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
      l = l * keep + lw;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] *= keep;
#pragma unroll 8
      for (int j = 0; j < here; ++j) {
        const float4 o = __ldcg(po + ((slot(k0 + j * 8) * 2 + tile) * (D / 4) + dims) * kChunkRows + in_tile);
        const float f = __shfl_sync(0xffffffffu, wa, j);
        if (f != 0.f) {  // a part without weight may hold anything
          acc[0] = fmaf(f, o.x, acc[0]), acc[1] = fmaf(f, o.y, acc[1]);
          acc[2] = fmaf(f, o.z, acc[2]), acc[3] = fmaf(f, o.w, acc[3]);
        }
      }
    }
    __syncthreads();
    float(*mine)[32] = shared_parts[warp];
    mine[4][lane] = m;
    mine[5][lane] = l;
#pragma unroll
    for (int j = 0; j < 4; ++j) mine[j][lane] = acc[j];
    __syncthreads();
    if (warp != 0) continue;
    for (int w = 1; w < 8; ++w) m = fmaxf(m, shared_parts[w][4][lane]);
    const float ref = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = 0.f;
    for (int w = 0; w < 8; ++w) {
      const float f = ex2_ftz(shared_parts[w][4][lane] - ref);
      l = fmaf(f, shared_parts[w][5][lane], l);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = fmaf(f, shared_parts[w][j][lane], acc[j]);
    }
    if (lane < kLanes) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const size_t at = ((size_t)(item.x + tok) * p.num_heads + cut.y * p.group + g) * D + 4 * lane;
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(static_cast<T*>(p.out) + at) =
            make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
      else
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at) =
            make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
    }
  }
}

// ---- host side ----

struct ChunkScratch {
  size_t cuts, part_ml, part_o, total;
};

ChunkScratch chunk_scratch(int head_size, int sm_count) {
  ChunkScratch s;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes, 256);
    return at;
  };
  const size_t rows = (size_t)2 * sm_count * 2 * kChunkRows;
  s.cuts = take(sizeof(int4) * (size_t)(2 * sm_count));
  s.part_ml = take(rows * 8);
  s.part_o = take(rows * head_size * 4);
  s.total = o;
  return s;
}

}  // namespace
}  // namespace pa
