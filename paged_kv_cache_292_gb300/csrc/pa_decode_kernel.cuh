// Paged decode attention for sm_103a.
//
// What it computes is section 3.2 ("内核执行流程（简化版）") of "vLLM
// three-process architecture and the PagedAttention kernel": for each
// sequence, look up its block table (step 1), bound the walk by its valid
// length (step 2), gather K/V from the scattered physical blocks (step 3),
// attend with the step's query (step 4) and write the output (step 5).  The
// same section's "精妙之处" asks for the gather to be planned up front and for
// copies to overlap compute on the GPU's separate copy engine; here that is
// two producer warps driving the TMA engine's copies into a ring of
// shared-memory stages while consumer warps compute on earlier stages.
//
// Kernel 1 (pa_decode_kernel), one CTA per (token range, KV-head group):
//   * The flattened tile list of the batch is cut into equal ranges (see
//     pa_schedule.h), so every CTA moves the same K/V bytes.
//   * The last two warps (the producers) walk the range tile by tile; both
//     follow every tile's bookkeeping and each takes alternate tiles: for a
//     tile of 16 tokens it looks up the block ids and copies K and V into the
//     tile's stage.
//     A token row is the `Hg` KV heads of the CTA's group, contiguous in the pool
//     ([block, slot, head, dim] layout), e.g. 2 KiB for 8 heads x 128 x bf16.
//     Tensor-core paths (bf16, FP8): one tensor-map box per run of
//     gcd(block_size, 16) rows of one block, landing with the 128-byte
//     swizzle in rows of an odd number of 128-byte lines (see RowPtr), so
//     ldmatrix reads of 8 consecutive tokens hit distinct banks.  fp32: one
//     bulk copy per token row, rows `row + 16` bytes apart.  Each sequence's
//     query slice is copied once into a small ring of its own.
//   * Each consumer warp owns one KV head and its G query heads (with several
//     query tokens and more than 8 (query, head) columns, two to four warps
//     share a KV head, 8 columns each).  bf16: S^T[16 tok x 8] = K_tile[16 x D] *
//     Q^T[D x 8] on the tensor cores (mma.sync m16n8k16, query heads padded
//     to 8), online softmax in registers (running max and sum in the exp2
//     domain), then O^T[D x 8] += V^T[D x 16] * P^T[16 x 8], with P^T obtained
//     from the score fragment by movmatrix.  FP8 pools: codes widened to f16
//     (MmaConsumerF8).  fp32: the same on CUDA cores.  FP8 consumers, and bf16
//     ones that share a KV head's columns with other warps, take two tiles of
//     one segment per pass when the ring has four or more stages (tile2).
//   * Appending calls also write the step's new tokens of each sequence: the
//     consumer warps put them into the staged tile and into the pool
//     (append_new_rows).  Not with several consumer warps per KV head, where
//     that code slowed the consumers' tile loop: the host then writes the rows
//     with a separate kernel ahead of the decode.
//   * Every wait is bounded; a wait that runs out sets PA_DEVERR_TIMEOUT, the
//     producers let the copies they started land before the CTA retires, and the
//     consumers take the tickets that they owe (give_up_tickets).
//   * A sequence wholly inside the range is written to `out` directly.  A
//     sequence cut by range boundaries leaves one (m, l, O) partial per range
//     and KV head; the warp that writes the last of them (an atomic ticket per
//     cut sequence and KV head, no waiting) then merges them all by log-sum-exp:
//     out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i.  The ticket counters
//     are reset by that warp, so the scratch is left zeroed for the next call.
//   * Empty sequences get zero output rows (all their query rows) from the
//     prologue.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include <type_traits>

#include "../../include/pagedattn.h"
#include "pa_device.cuh"
#include "pa_layout.h"
#include "pa_schedule.h"

namespace pa {

enum : int { kSegBegin = 1, kSegEnd = 2 };

struct StageMeta {
  int seq;     // sequence index
  int tok0;    // first token of the tile within the sequence
  int nvalid;  // valid tokens in the tile (1..16); kWalkMod: bit mask of the rows some query sees
  int flags;   // kSegBegin | kSegEnd | (output slot + 1) << 2 | (slot of range r0) << 4 | tile_tag
  int r0, r1;  // first and last range touching the sequence (cut sequences only)
  int ctx;     // the sequence's context length (causal limits of several queries)
  int newfirst;  // appending calls: first tile row holding one of the step's new
                 // tokens (rows newfirst .. nvalid-1; their pool rows are in the
                 // stage's row list); -1 when the tile holds none.  kWalkMod:
                 // tokens before this one are seen by every query
};

struct DecodeParams {
  CUtensorMap tm_k, tm_v;  // tensor-core paths: 4-D views of the pools (see make_tensor_maps)
  void* out;
  // Appending calls (bf16, at most 8 (query, head) columns per KV head): K/V
  // rows [num_seqs * num_queries, num_kv_heads, head_size] of each sequence's
  // new tokens (row s * Q + i: position c - Q + i), written into the pool by
  // the decode itself; nullptr otherwise.
  const void* k_new;
  const void* v_new;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* counters;  // [num_ranges - 1][num_kv_heads] merge tickets (of the sequence that a range's end cuts); zero between calls
  float* part_ml;   // [R][2][H][2]: (m in log2 units, l)
  float* part_o;    // [R][2][H][D]: un-normalised weighted V sums
  int32_t* error_flag;
  int num_seqs, num_heads, num_kv_heads, group, block_size, max_blocks_per_seq;
  int heads_per_cta;    // Hg
  int num_head_groups;  // HG = Hk / Hg
  int num_ranges;       // R
  int num_physical_blocks;
  int stages, q_slots;
  int num_queries;  // query tokens per sequence (1 for plain decode)
  int split;        // consumer warps per KV head: ceil(G * num_queries / 8), 8 columns each
  float v_scale;    // FP8 pools: value of a V code is decode(code) * v_scale (else 1)
  float k_scale;    // FP8 pools: value of a K code is decode(code) * k_scale (else 1)
  uint32_t row_bytes, pitch, q_bytes, stage_bytes;
  uint32_t lines;      // tensor-core stages: 128-byte lines per staged token row
  uint32_t box_rows;   // token rows per tensor copy: gcd(block_size, 16)
  uint32_t box_bytes;  // bytes one tensor copy lands (box_rows * lines * 128)
  float scale_log2;    // scale * log2(e)
  // Modified scores (kWalkMod): s = cap * tanh(scale * q.k / cap), then
  // - slope * |distance|; visibility by window, first token and prefix.
  float cap_in;   // tensor-core paths: 2 * log2(e) * scale / cap, the base-2 exponent of
                  // tanh's e^2x; fp32: scale / cap
  float cap_out;  // cap * log2(e); 0: scores are not capped
  const float* slopes;          // [num_heads] or nullptr
  const int32_t* first_tokens;  // [num_seqs] or nullptr
  const int32_t* prefix_lens;   // [num_seqs] or nullptr
  int window;                   // tokens a query sees back from its own position (kNoWindow: all)
  // Rest of a shared prefix (kWalkRest): sequences of at least
  // prefix_tokens + num_queries - 1 tokens are walked from prefix_tokens on, the others
  // whole; (m, l) and un-normalised O of every row go to rest_ml / rest_o.
  int prefix_tokens;
  // Both: how each sequence was cut (see SeqCut); the partials are merged by a
  // kernel behind this one, all rows at once.
  int4* cuts;
  int sm_count;
  // kWalkRest behind the prefix kernel: the grid starts beside it (its CTAs have
  // let this one go, so what came before both is complete) and only its end
  // waits for it.  prefix_units: that kernel's work, for sharing out the SMs.
  bool beside;
  float prefix_units;
  float* rest_ml;  // [num_seqs * num_queries * num_heads][2]
  float* rest_o;   // [num_seqs * num_queries * num_heads][D]
  // int8 pools: a scale for every token and KV head, [block][KV head][row of the block]; in a stage
  // they lie behind K and V: [K, V][head of the group][16].
  const float* k_scales;
  const float* v_scales;
  unsigned long long wait_limit_ns;  // bound of every pipeline wait
  long long stall_tile;  // tests of the bounded waits: flattened tile whose copies are withheld (-1: none)
};

__device__ __forceinline__ int clamp_context(const DecodeParams& p, int s, bool report_it) {
  int c = __ldg(p.context_lens + s);
  const int cmax = p.max_blocks_per_seq * p.block_size;
  if (c < 0 || c > cmax) {
    if (report_it) report(p.error_flag, PA_DEVERR_CONTEXT_LEN);
    c = c < 0 ? 0 : cmax;
  }
  return c;
}

// Sequence s as the walk takes it (SeqSpan).
template <int WALK>
struct SeqWalk : SeqSpan<WALK> {
  __device__ __forceinline__ SeqWalk() {}
  __device__ __forceinline__ SeqWalk(const DecodeParams& p, int s, bool report_it) {
    const int context = clamp_context(p, s, report_it);
    if constexpr (WALK == kWalkAll) {
      this->all(context);
    } else if constexpr (WALK == kWalkRest) {
      this->rest(context, p.prefix_tokens, p.num_queries);
    } else {
      this->seen(context, p.first_tokens != nullptr ? __ldg(p.first_tokens + s) : 0,
                 p.prefix_lens != nullptr ? __ldg(p.prefix_lens + s) : 0, p.num_queries, p.window);
    }
  }
};

// SMs for the prefix kernel of `units` units (pa_prefix_work.h) beside a walk of
// `tiles` tiles by `groups` CTAs each, in proportion to the SM time of either: a
// unit takes about 0.9 us (D = 128: 128 x 128 x 128 x 4 flops; D = 64: 0.78, where the
// softmax sets the pace), a tile about 0.35 us + 0.18 us per KiB of K row, or 0.8 us with
// more than 8 columns per KV head, and a sequence another 0.8 us per 4096 elements of
// its query and output rows (0.8 to 2.4).  The walk is bound by HBM from about 80 SMs on.
//   256 sequences of 64 heads with a tile each behind 32k tokens: 253 us, with 0.8 us
// for any sequence 359 (the walk came last); of 32 heads on 16k: 83, with 1.6 us 86.
__device__ __forceinline__ int prefix_share(float units, long long tiles, int seqs, int groups, float tile_us,
                                            int row_elements, int head_size, int sm_count) {
  if (tiles == 0) return sm_count;
  const float seq_us = 0.8f * fminf(fmaxf(row_elements * (1.f / 4096.f), 1.f), 3.f);
  const float a = units * (head_size == 128 ? 0.9f : 0.78f), b = (tiles * tile_us + seqs * seq_us) * groups;
  // The walk's part in whole ranges (one CTA per group of KV heads each).
  const int walk = (__float2int_ru(sm_count * (b / (a + b))) + groups - 1) / groups * groups;
  return max(1, sm_count - max(walk, groups));
}
__device__ __forceinline__ float walk_tile_us(uint32_t row_bytes, int columns) {
  return columns > 8 ? 0.8f : 0.35f + 0.18f / 1024.f * row_bytes;
}

__device__ __forceinline__ long long warp_sum_ll(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ long long warp_incl_scan_ll(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    long long n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// ---------------------------------------------------------------------------
// Consumer state and tile math.  One consumer warp = one KV head and its G
// query heads; D = head size.
// ---------------------------------------------------------------------------

// Stages of the tensor-core consumers.  A K or V half-stage holds the tile's
// 16 token rows, row r as `lines` 128-byte lines (the head group's bytes,
// then zero-filled lines up to an odd count or the count a copy's alignment
// needs), written by tensor copies with the 128-byte swizzle: line
// L = r * lines + chunk stores its 16-byte unit u at position u ^ (L % 8).
// With `lines` odd, one unit of 8 consecutive rows lands in 8 different bank
// groups, so ldmatrix reads are conflict-free.
//
// RowPtr<NC> holds one lane's ldmatrix row address for a head whose bytes
// span NC 128-byte chunks: units u0 + 2j (j = 0, 1, ...) of row r, where u0
// counts 16-byte units from the start of the group's row and has bits 1-2
// clear, so stepping j within a chunk flips address bits 5-6 only.
template <int NC>
struct RowPtr {
  uint32_t a[NC];
  __device__ __forceinline__ RowPtr(uint32_t half, int r, int u0, uint32_t lines) {
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint32_t unit = (uint32_t)u0 + 8u * c;
      const uint32_t L = (uint32_t)r * lines + (unit >> 3);
      a[c] = half + L * kLine + (((unit & 7u) ^ (L & 7u)) << 4);
    }
  }
  __device__ __forceinline__ uint32_t at(int j) const { return a[j >> 2] ^ ((uint32_t)(j & 3) << 5); }
};

// Modified scores of one 16-token tile.  A lane holds rows r0 and r0 + 8 of
// columns a and b, as (row r0: a, b; row r0 + 8: a, b).
struct ModTile {
  uint32_t vis;  // rows some query of the sequence sees
  int tok0, ctx;
  int pre;  // tokens before this one are seen by every query
};

struct ModCols {
  int qa = 0, qb = 0;        // query index of each column (padding columns: any)
  float sa = 0.f, sb = 0.f;  // log2(e) * slope of each column's head

  // n: column a of (query, head) columns n = query * G + head, column b the next.
  __device__ __forceinline__ void setup(const DecodeParams& p, int kv_head, int n) {
    const int G = p.group, Q = p.num_queries;
    qa = n < G * Q ? n / G : 0;
    qb = n + 1 < G * Q ? (n + 1) / G : 0;
    if (p.slopes != nullptr) {
      if (n < G * Q) sa = 1.4426950408889634f * __ldg(p.slopes + kv_head * G + n % G);
      if (n + 1 < G * Q) sb = 1.4426950408889634f * __ldg(p.slopes + kv_head * G + (n + 1) % G);
    }
  }
};

// x -> capped scores in log2 units.  tanh(t) = 1 - 2 / (1 + e^2t) runs on the SFU
// (one 2^x, one reciprocal), with an absolute error of up to 2^-22 of the cap: 2^-16
// of a score's unit at kSfuCap = 64, far below the rounding of the bf16 output.
//   Larger caps take the series t (1 - t^2/3 + 2 t^4/15 - 17 t^6/315) below t = 1/8
// (relative error 2^-29), its factor on the uncapped score, so that a cap too large for any
// score changes nothing.  With it for all caps 48 sequences x 4 queries over FP8
// pools take 61 us, without it 56.
constexpr float kSfuCap = 64.f * 1.4426950408889634f;  // in log2 units

__device__ __forceinline__ float cap_sfu(const DecodeParams& p, float y) {
  return p.cap_out - 2.f * p.cap_out * rcp_ftz(1.f + ex2_ftz(y));
}

template <int N>
__device__ __forceinline__ void cap_scores(const DecodeParams& p, float (&x)[N]) {
  if (p.cap_out == 0.f) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] *= p.scale_log2;
  } else if (p.cap_out <= kSfuCap) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = cap_sfu(p, x[i] * p.cap_in);
  } else {
    constexpr float kT = 0.34657359f, kT2 = kT * kT;  // t = kT y: ln 2 / 2
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = x[i] * p.cap_in, y2 = y * y;
      const float f =
          fmaf(fmaf(fmaf(-17.f / 315.f * kT2 * kT2 * kT2, y2, 2.f / 15.f * kT2 * kT2), y2, -kT2 / 3.f), y2, 1.f);
      x[i] = fabsf(y) < 0.125f / kT ? x[i] * p.scale_log2 * f : cap_sfu(p, y);
    }
  }
}

__device__ __forceinline__ void mod_scores(const DecodeParams& p, const ModCols& mc, const ModTile& t, int r0,
                                           float& s0, float& s1, float& s2, float& s3) {
  float x[4] = {s0, s1, s2, s3};
  cap_scores(p, x);
  s0 = x[0], s1 = x[1], s2 = x[2], s3 = x[3];
  const int base = t.ctx - p.num_queries, row = t.tok0 + r0;
  if (p.slopes != nullptr) {
    const float da = static_cast<float>(base + mc.qa - row), db = static_cast<float>(base + mc.qb - row);
    s0 -= mc.sa * fabsf(da);
    s1 -= mc.sb * fabsf(db);
    s2 -= mc.sa * fabsf(da - 8.f);
    s3 -= mc.sb * fabsf(db - 8.f);
  }
  // Do all queries see all rows?  (The same answer for the whole warp.)
  const bool split = base < 0 || (t.tok0 + kTile > t.pre &&
                                  (t.tok0 + kTile - 1 > base || t.tok0 <= t.ctx - 1 - p.window));
  if (split) {
    const int pa = base + mc.qa, pb = base + mc.qb;
    const int la = pa - p.window, lb = pb - p.window;
    const bool pre0 = row < t.pre, pre1 = row + 8 < t.pre;
    if (pa < 0 || !(pre0 || (row <= pa && row > la))) s0 = -INFINITY;
    if (pb < 0 || !(pre0 || (row <= pb && row > lb))) s1 = -INFINITY;
    if (pa < 0 || !(pre1 || (row + 8 <= pa && row + 8 > la))) s2 = -INFINITY;
    if (pb < 0 || !(pre1 || (row + 8 <= pb && row + 8 > lb))) s3 = -INFINITY;
  }
  if (t.vis != 0xffffu) {
    if (!((t.vis >> r0) & 1u)) s0 = s1 = -INFINITY;
    if (!((t.vis >> (r0 + 8)) & 1u)) s2 = s3 = -INFINITY;
  }
}

// The same for the row form (RowsConsumer): a lane holds columns t2, t2 + 1, t2 + 8,
// t2 + 9 (tokens) of rows a (s[0..3]) and b (s[4..7]).  Without MOD: plain scores
// under the causal mask.
template <bool MOD>
__device__ __forceinline__ void row_scores(const DecodeParams& p, const ModCols& mc, const ModTile& t, int t2,
                                           float (&s)[8]) {
  const int base = t.ctx - p.num_queries, col = t.tok0 + t2;
  const int pa = base + mc.qa, pb = base + mc.qb;
  if constexpr (MOD) {
    cap_scores(p, s);
    if (p.slopes != nullptr) {
      const float da = static_cast<float>(pa - col), db = static_cast<float>(pb - col);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float d = static_cast<float>((i & 1) + 8 * (i >> 1));
        s[i] -= mc.sa * fabsf(da - d);
        s[4 + i] -= mc.sb * fabsf(db - d);
      }
    }
    // Do all queries see all tokens?  (The same answer for the whole warp.)
    if (base < 0 || (t.tok0 + kTile > t.pre && (t.tok0 + kTile - 1 > base || t.tok0 <= t.ctx - 1 - p.window))) {
      const int la = pa - p.window, lb = pb - p.window;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = col + (i & 1) + 8 * (i >> 1);
        const bool pre = c < t.pre;
        if (pa < 0 || !(pre || (c <= pa && c > la))) s[i] = -INFINITY;
        if (pb < 0 || !(pre || (c <= pb && c > lb))) s[4 + i] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] *= p.scale_log2;
    if (t.tok0 + kTile > base) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = col + (i & 1) + 8 * (i >> 1);
        if (c > pa) s[i] = -INFINITY;
        if (c > pb) s[4 + i] = -INFINITY;
      }
    }
  }
  if (t.vis != 0xffffu) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!((t.vis >> (t2 + (i & 1) + 8 * (i >> 1))) & 1u)) s[i] = s[4 + i] = -INFINITY;
  }
}

// Halves of a V fragment register (tokens t2, t2 + 1) to keep.
__device__ __forceinline__ uint32_t keep_pair(uint32_t vis, int t2) {
  return ((vis >> t2) & 1u ? 0x0000ffffu : 0u) | ((vis >> (t2 + 1)) & 1u ? 0xffff0000u : 0u);
}

// bf16 tensor-core consumer.  Lane l owns query heads hA = 2*(l%4), hB = hA+1
// (columns of the score fragment) and, per 16-wide slice mt of the head
// dimension, output dims mt*16 + l/4 and +8.
template <int D>
struct MmaConsumer {
  static constexpr int KS = D / 16;  // k-steps of Q.K and m-tiles of P.V
  uint32_t qb[KS][2];
  float acc[KS][4];
  float m_a, m_b, l_a, l_b;

  __device__ __forceinline__ void begin_segment(const unsigned char* qslot, int w, int G,
                                                int lane) {
    const int n = lane >> 2, t2 = 2 * (lane & 3);
    const __nv_bfloat16* qh =
        reinterpret_cast<const __nv_bfloat16*>(qslot) + (size_t)(w * G + n) * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (n < G) {
        qb[ks][0] = *reinterpret_cast<const uint32_t*>(qh + ks * 16 + t2);
        qb[ks][1] = *reinterpret_cast<const uint32_t*>(qh + ks * 16 + 8 + t2);
      } else {
        qb[ks][0] = 0u;
        qb[ks][1] = 0u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[ks][i] = 0.f;
    }
    m_a = m_b = -INFINITY;
    l_a = l_b = 0.f;
  }

  static constexpr int NC = D * 2 > 128 ? D * 2 / 128 : 1;  // 128-byte chunks per head

  // k_half / v_half: the stage's K and V halves; uh: first 16-byte unit of
  // this warp's head within the group's row.
  __device__ __forceinline__ void tile(uint32_t k_half, uint32_t v_half, uint32_t lines, int uh,
                                       int nvalid, float scale_log2, int lane) {
    // S^T = K_tile * Q^T : rows = tokens, columns = query heads.
    float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
    const RowPtr<NC> kp(k_half, (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), lines);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[4];
      ldmatrix_x4(a, kp.at(ks));
      if (ks & 1)
        mma_bf16_16816(c1, a, qb[ks][0], qb[ks][1]);
      else
        mma_bf16_16816(c0, a, qb[ks][0], qb[ks][1]);
    }
    const int r0 = lane >> 2;
    float s0 = (c0[0] + c1[0]) * scale_log2, s1 = (c0[1] + c1[1]) * scale_log2;
    float s2 = (c0[2] + c1[2]) * scale_log2, s3 = (c0[3] + c1[3]) * scale_log2;
    if (r0 >= nvalid) s0 = s1 = -INFINITY;
    if (r0 + 8 >= nvalid) s2 = s3 = -INFINITY;

    // Online softmax: per-head tile maximum across the 8 lanes sharing l%4.
    float mx_a = fmaxf(s0, s2), mx_b = fmaxf(s1, s3);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
    }
    const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
    // A tile always holds a valid token, so mn_* is finite unless the inputs
    // are not; guard the exponent base anyway so -inf - -inf never appears.
    const float base_a = (mn_a == -INFINITY) ? 0.f : mn_a;
    const float base_b = (mn_b == -INFINITY) ? 0.f : mn_b;
    const float alpha_a = ex2_ftz(m_a - base_a), alpha_b = ex2_ftz(m_b - base_b);
    m_a = mn_a;
    m_b = mn_b;
    const float p0 = ex2_ftz(s0 - base_a), p1 = ex2_ftz(s1 - base_b);
    const float p2 = ex2_ftz(s2 - base_a), p3 = ex2_ftz(s3 - base_b);
    // P enters the bf16 MMA as a high and a low bf16 part (P = hi + lo to
    // about 2^-16), so the weights keep fp32-like precision.
    const uint32_t p_top = pack_bf16x2(p0, p1), p_bot = pack_bf16x2(p2, p3);
    const uint32_t r_top = pack_bf16x2(p0 - bf16_lo(p_top), p1 - bf16_hi(p_top));
    const uint32_t r_bot = pack_bf16x2(p2 - bf16_lo(p_bot), p3 - bf16_hi(p_bot));
    l_a = l_a * alpha_a + p0 + p2;
    l_b = l_b * alpha_b + p1 + p3;
    const uint32_t pb0 = movmatrix_trans(p_top);  // P^T rows (tokens) 0-7
    const uint32_t pb1 = movmatrix_trans(p_bot);  // tokens 8-15
    const uint32_t rb0 = movmatrix_trans(r_top);
    const uint32_t rb1 = movmatrix_trans(r_bot);

    // O^T += V^T * P^T : rows = head dims, columns = query heads.
    const RowPtr<NC> vp(v_half, (lane & 7) + (lane >> 4) * 8, uh + ((lane >> 3) & 1), lines);
    const int t2 = 2 * (lane & 3);
    uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
    if (nvalid < kTile) {
      // Zero V entries of tokens past the end so stale stage contents (which
      // may be non-finite) never meet a zero weight.
      keep_lo = (t2 < nvalid ? 0x0000ffffu : 0u) | (t2 + 1 < nvalid ? 0xffff0000u : 0u);
      keep_hi = (t2 + 8 < nvalid ? 0x0000ffffu : 0u) | (t2 + 9 < nvalid ? 0xffff0000u : 0u);
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t a[4];
      ldmatrix_x4_trans(a, vp.at(mt));
      a[0] &= keep_lo;
      a[1] &= keep_lo;
      a[2] &= keep_hi;
      a[3] &= keep_hi;
      acc[mt][0] *= alpha_a;
      acc[mt][1] *= alpha_b;
      acc[mt][2] *= alpha_a;
      acc[mt][3] *= alpha_b;
      mma_bf16_16816(acc[mt], a, pb0, pb1);
      mma_bf16_16816(acc[mt], a, rb0, rb1);
    }
  }

  // slot < 0: final output (REST: the row's (m, l, O)); else partial slot of range r.
  template <bool REST = false>
  __device__ __forceinline__ void finish(const DecodeParams& p, int seq, int kv_head, int slot,
                                         int r, int lane) {
    float la = l_a, lb = l_b;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      la += __shfl_xor_sync(0xffffffffu, la, o);
      lb += __shfl_xor_sync(0xffffffffu, lb, o);
    }
    const int G = p.group, H = p.num_heads;
    const int ha = 2 * (lane & 3), hb = ha + 1, d0 = lane >> 2;
    const int qa = kv_head * G + ha, qb_ = kv_head * G + hb;
    if (!REST && slot < 0) {
      __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + (size_t)seq * H * D;
      const float ia = 1.f / la, ib = 1.f / lb;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int d = mt * 16 + d0;
        if (ha < G) {
          out[(size_t)qa * D + d] = __float2bfloat16_rn(acc[mt][0] * ia);
          out[(size_t)qa * D + d + 8] = __float2bfloat16_rn(acc[mt][2] * ia);
        }
        if (hb < G) {
          out[(size_t)qb_ * D + d] = __float2bfloat16_rn(acc[mt][1] * ib);
          out[(size_t)qb_ * D + d + 8] = __float2bfloat16_rn(acc[mt][3] * ib);
        }
      }
    } else {
      const bool whole = REST && slot < 0;
      const size_t base = whole ? (size_t)seq * H : ((size_t)r * 2 + slot) * H;
      float* po = (whole ? p.rest_o : p.part_o) + base * D;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const int d = mt * 16 + d0;
        if (ha < G) {
          po[(size_t)qa * D + d] = acc[mt][0];
          po[(size_t)qa * D + d + 8] = acc[mt][2];
        }
        if (hb < G) {
          po[(size_t)qb_ * D + d] = acc[mt][1];
          po[(size_t)qb_ * D + d + 8] = acc[mt][3];
        }
      }
      if (d0 == 0) {
        float* pm = (whole ? p.rest_ml : p.part_ml) + base * 2;
        if (ha < G) {
          pm[(size_t)qa * 2 + 0] = m_a;
          pm[(size_t)qa * 2 + 1] = la;
        }
        if (hb < G) {
          pm[(size_t)qb_ * 2 + 0] = m_b;
          pm[(size_t)qb_ * 2 + 1] = lb;
        }
      }
    }
  }
};

// bf16 tensor-core consumer for several query tokens per sequence (causal).
// The N extent of the score fragment holds (query, head) columns: column
// n = qi * G + g for query qi < Q and group head g < G, NT tiles of 8 columns.
// Query qi sits at position ctx - Q + qi and sees tokens up to that position.
// MOD: modified scores (mod_scores) instead of the causal mask alone; `mo` is
// the tile's mask and position.
template <int D, int NT, bool MOD = false>
struct MmaConsumerMQ {
  static constexpr int KS = D / 16;
  uint32_t qb[NT][KS][2];
  float acc[NT][KS][4];
  float m_a[NT], m_b[NT], l_a[NT], l_b[NT];
  int col0 = 0;  // first (query, head) column this warp owns
  ModCols mc;    // MOD

  // w: KV head within the CTA's group; col_base: first column of this warp.
  __device__ __forceinline__ void begin_segment(const unsigned char* qslot, int w, int G, int Q,
                                                int Hg, int lane, int col_base) {
    col0 = col_base;
    const int t2 = 2 * (lane & 3);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = col0 + nt * 8 + (lane >> 2);
      const bool real = n < G * Q;
      const int qi = real ? n / G : 0, g = real ? n % G : 0;
      const __nv_bfloat16* qh =
          reinterpret_cast<const __nv_bfloat16*>(qslot) + ((size_t)qi * Hg * G + w * G + g) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[nt][ks][0] = real ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + t2) : 0u;
        qb[nt][ks][1] = real ? *reinterpret_cast<const uint32_t*>(qh + ks * 16 + 8 + t2) : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][ks][i] = 0.f;
      }
      m_a[nt] = m_b[nt] = -INFINITY;
      l_a[nt] = l_b[nt] = 0.f;
    }
  }

  // After a segment's finish (and merge) every state register is rewritten
  // by the next begin_segment before it is read; writing them here tells the
  // compiler so, which frees them for the merge.
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        qb[nt][ks][0] = qb[nt][ks][1] = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][ks][i] = 0.f;
      }
      m_a[nt] = m_b[nt] = l_a[nt] = l_b[nt] = 0.f;
    }
  }

  static constexpr int NC = D * 2 > 128 ? D * 2 / 128 : 1;

  __device__ __forceinline__ void tile(uint32_t k_half, uint32_t v_half, uint32_t lines, int uh,
                                       int nvalid, int tok0, int ctx, int G, int Q,
                                       float scale_log2, int lane, const DecodeParams* mod = nullptr,
                                       const ModTile& mo = ModTile()) {
    // Scores accumulate in two independent chains (even / odd k-steps) that
    // are added at the end: with one 8-column tile per warp, a single chain
    // would serialise all KS MMAs.
    float c[NT][4], c2[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[nt][i] = c2[nt][i] = 0.f;
    const RowPtr<NC> kp(k_half, (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), lines);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a[4];
      ldmatrix_x4(a, kp.at(ks));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816((ks & 1) ? c2[nt] : c[nt], a, qb[nt][ks][0], qb[nt][ks][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[nt][i] += c2[nt][i];
    const int r0 = lane >> 2;
    const int t0 = tok0 + r0, t1 = t0 + 8;
    uint32_t pb0[NT], pb1[NT], rb0[NT], rb1[NT];
    float alpha_a[NT], alpha_b[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float s0 = c[nt][0], s1 = c[nt][1], s2 = c[nt][2], s3 = c[nt][3];
      if constexpr (MOD) {
        mod_scores(*mod, mc, mo, r0, s0, s1, s2, s3);
      } else {
        s0 *= scale_log2;
        s1 *= scale_log2;
        s2 *= scale_log2;
        s3 *= scale_log2;
        if (r0 >= nvalid) s0 = s1 = -INFINITY;
        if (r0 + 8 >= nvalid) s2 = s3 = -INFINITY;
        // Causal limits matter only on tiles that reach the queries' own
        // positions (ctx - Q ..); the test is the same for the whole warp.
        if (tok0 + kTile > ctx - Q) {
          const int na = col0 + nt * 8 + 2 * (lane & 3), nb = na + 1;
          // Last visible position of each column's query (-1: padding column).
          const int lim_a = na < G * Q ? ctx - Q + na / G : -1;
          const int lim_b = nb < G * Q ? ctx - Q + nb / G : -1;
          if (t0 > lim_a) s0 = -INFINITY;
          if (t0 > lim_b) s1 = -INFINITY;
          if (t1 > lim_a) s2 = -INFINITY;
          if (t1 > lim_b) s3 = -INFINITY;
        }
      }
      float mx_a = fmaxf(s0, s2), mx_b = fmaxf(s1, s3);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
      }
      const float mn_a = fmaxf(m_a[nt], mx_a), mn_b = fmaxf(m_b[nt], mx_b);
      // A column may see no token of this tile (or none yet): keep -inf out of
      // the exponent base.
      const float base_a = (mn_a == -INFINITY) ? 0.f : mn_a;
      const float base_b = (mn_b == -INFINITY) ? 0.f : mn_b;
      alpha_a[nt] = ex2_ftz(m_a[nt] - base_a);
      alpha_b[nt] = ex2_ftz(m_b[nt] - base_b);
      m_a[nt] = mn_a;
      m_b[nt] = mn_b;
      const float p0 = ex2_ftz(s0 - base_a), p1 = ex2_ftz(s1 - base_b);
      const float p2 = ex2_ftz(s2 - base_a), p3 = ex2_ftz(s3 - base_b);
      const uint32_t p_top = pack_bf16x2(p0, p1), p_bot = pack_bf16x2(p2, p3);
      const uint32_t r_top = pack_bf16x2(p0 - bf16_lo(p_top), p1 - bf16_hi(p_top));
      const uint32_t r_bot = pack_bf16x2(p2 - bf16_lo(p_bot), p3 - bf16_hi(p_bot));
      l_a[nt] = l_a[nt] * alpha_a[nt] + p0 + p2;
      l_b[nt] = l_b[nt] * alpha_b[nt] + p1 + p3;
      pb0[nt] = movmatrix_trans(p_top);
      pb1[nt] = movmatrix_trans(p_bot);
      rb0[nt] = movmatrix_trans(r_top);
      rb1[nt] = movmatrix_trans(r_bot);
    }
    const RowPtr<NC> vp(v_half, (lane & 7) + (lane >> 4) * 8, uh + ((lane >> 3) & 1), lines);
    const int t2 = 2 * (lane & 3);
    uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
    if constexpr (MOD) {
      if (mo.vis != 0xffffu) {
        keep_lo = keep_pair(mo.vis, t2);
        keep_hi = keep_pair(mo.vis, t2 + 8);
      }
    } else if (nvalid < kTile) {
      keep_lo = (t2 < nvalid ? 0x0000ffffu : 0u) | (t2 + 1 < nvalid ? 0xffff0000u : 0u);
      keep_hi = (t2 + 8 < nvalid ? 0x0000ffffu : 0u) | (t2 + 9 < nvalid ? 0xffff0000u : 0u);
    }
    // Rescale the accumulators only when some running max moved (a warp vote).
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) moved |= (alpha_a[nt] != 1.f) || (alpha_b[nt] != 1.f);
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][mt][0] *= alpha_a[nt];
          acc[nt][mt][1] *= alpha_b[nt];
          acc[nt][mt][2] *= alpha_a[nt];
          acc[nt][mt][3] *= alpha_b[nt];
        }
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t a[4];
      ldmatrix_x4_trans(a, vp.at(mt));
      a[0] &= keep_lo;
      a[1] &= keep_lo;
      a[2] &= keep_hi;
      a[3] &= keep_hi;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_bf16_16816(acc[nt][mt], a, pb0[nt], pb1[nt]);
        mma_bf16_16816(acc[nt][mt], a, rb0[nt], rb1[nt]);
      }
    }
  }

  // The same with all K fragments loaded first, the scores in four chains
  // and the V fragments loaded before the softmax (used when a KV head's
  // columns are split over several warps, where it measured faster).
  __device__ __forceinline__ void tile_hoisted(uint32_t k_half, uint32_t v_half, uint32_t lines, int uh,
                                               int nvalid, int tok0, int ctx, int G, int Q,
                                       float scale_log2, int lane) {
    // All K fragments are loaded first, then the scores accumulate in four
    // independent chains (k-step mod 4) added at the end: with one 8-column
    // tile per warp a single chain would serialise all KS MMAs.  The V
    // fragments are loaded right after, so their latency overlaps the softmax.
    constexpr int NCH = KS < 4 ? KS : 4;
    uint32_t kf[KS][4], vf[KS][4];
    const RowPtr<NC> kp(k_half, (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), lines);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) ldmatrix_x4(kf[ks], kp.at(ks));
    float cc[NCH][NT][4];
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) cc[ch][nt][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(cc[ks % NCH][nt], kf[ks], qb[nt][ks][0], qb[nt][ks][1]);
    const RowPtr<NC> vp(v_half, (lane & 7) + (lane >> 4) * 8, uh + ((lane >> 3) & 1), lines);
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) ldmatrix_x4_trans(vf[mt], vp.at(mt));
    float c[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = cc[0][nt][i];
#pragma unroll
        for (int ch = 1; ch < NCH; ++ch) v += cc[ch][nt][i];
        c[nt][i] = v;
      }
    const int r0 = lane >> 2;
    const int t0 = tok0 + r0, t1 = t0 + 8;
    uint32_t pb0[NT], pb1[NT], rb0[NT], rb1[NT];
    float alpha_a[NT], alpha_b[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float s0 = c[nt][0] * scale_log2, s1 = c[nt][1] * scale_log2;
      float s2 = c[nt][2] * scale_log2, s3 = c[nt][3] * scale_log2;
      if (r0 >= nvalid) s0 = s1 = -INFINITY;
      if (r0 + 8 >= nvalid) s2 = s3 = -INFINITY;
      // Causal limits matter only on tiles that reach the queries' own
      // positions (ctx - Q ..); the test is the same for the whole warp.
      if (tok0 + kTile > ctx - Q) {
        const int na = col0 + nt * 8 + 2 * (lane & 3), nb = na + 1;
        // Last visible position of each column's query (-1: padding column).
        const int lim_a = na < G * Q ? ctx - Q + na / G : -1;
        const int lim_b = nb < G * Q ? ctx - Q + nb / G : -1;
        if (t0 > lim_a) s0 = -INFINITY;
        if (t0 > lim_b) s1 = -INFINITY;
        if (t1 > lim_a) s2 = -INFINITY;
        if (t1 > lim_b) s3 = -INFINITY;
      }
      float mx_a = fmaxf(s0, s2), mx_b = fmaxf(s1, s3);
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
      }
      const float mn_a = fmaxf(m_a[nt], mx_a), mn_b = fmaxf(m_b[nt], mx_b);
      // A column may see no token of this tile (or none yet): keep -inf out of
      // the exponent base.
      const float base_a = (mn_a == -INFINITY) ? 0.f : mn_a;
      const float base_b = (mn_b == -INFINITY) ? 0.f : mn_b;
      alpha_a[nt] = ex2_ftz(m_a[nt] - base_a);
      alpha_b[nt] = ex2_ftz(m_b[nt] - base_b);
      m_a[nt] = mn_a;
      m_b[nt] = mn_b;
      const float p0 = ex2_ftz(s0 - base_a), p1 = ex2_ftz(s1 - base_b);
      const float p2 = ex2_ftz(s2 - base_a), p3 = ex2_ftz(s3 - base_b);
      const uint32_t p_top = pack_bf16x2(p0, p1), p_bot = pack_bf16x2(p2, p3);
      const uint32_t r_top = pack_bf16x2(p0 - bf16_lo(p_top), p1 - bf16_hi(p_top));
      const uint32_t r_bot = pack_bf16x2(p2 - bf16_lo(p_bot), p3 - bf16_hi(p_bot));
      l_a[nt] = l_a[nt] * alpha_a[nt] + p0 + p2;
      l_b[nt] = l_b[nt] * alpha_b[nt] + p1 + p3;
      pb0[nt] = movmatrix_trans(p_top);
      pb1[nt] = movmatrix_trans(p_bot);
      rb0[nt] = movmatrix_trans(r_top);
      rb1[nt] = movmatrix_trans(r_bot);
    }
    const int t2 = 2 * (lane & 3);
    uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
    if (nvalid < kTile) {
      keep_lo = (t2 < nvalid ? 0x0000ffffu : 0u) | (t2 + 1 < nvalid ? 0xffff0000u : 0u);
      keep_hi = (t2 + 8 < nvalid ? 0x0000ffffu : 0u) | (t2 + 9 < nvalid ? 0xffff0000u : 0u);
    }
    // Rescale the accumulators only when some running max moved (a warp vote).
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) moved |= (alpha_a[nt] != 1.f) || (alpha_b[nt] != 1.f);
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][mt][0] *= alpha_a[nt];
          acc[nt][mt][1] *= alpha_b[nt];
          acc[nt][mt][2] *= alpha_a[nt];
          acc[nt][mt][3] *= alpha_b[nt];
        }
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      vf[mt][0] &= keep_lo;
      vf[mt][1] &= keep_lo;
      vf[mt][2] &= keep_hi;
      vf[mt][3] &= keep_hi;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(acc[nt][mt], vf[mt], pb0[nt], pb1[nt]);
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(acc[nt][mt], vf[mt], rb0[nt], rb1[nt]);
  }

  // Two consecutive tiles of one segment in one pass (the first full, from
  // tok0; the second with nvalid1 tokens from tok0 + 16): the two tiles'
  // score chains interleave and one softmax update covers all 32 tokens.
  __device__ __forceinline__ void tile2(uint32_t k_half0, uint32_t v_half0, uint32_t k_half1, uint32_t v_half1,
                                        uint32_t lines, int uh, int nvalid1, int tok0, int ctx, int G, int Q,
                                        float scale_log2, int lane) {
    const RowPtr<NC> kp0(k_half0, (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), lines);
    const RowPtr<NC> kp1(k_half1, (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), lines);
    float cc[2][2][NT][4];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int ch = 0; ch < 2; ++ch)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) cc[tt][ch][nt][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      uint32_t a0[4], a1[4];
      ldmatrix_x4(a0, kp0.at(ks));
      ldmatrix_x4(a1, kp1.at(ks));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_bf16_16816(cc[0][ks & 1][nt], a0, qb[nt][ks][0], qb[nt][ks][1]);
        mma_bf16_16816(cc[1][ks & 1][nt], a1, qb[nt][ks][0], qb[nt][ks][1]);
      }
    }
    const int r0 = lane >> 2;
    uint32_t pb[2][NT][4];  // per tile: P^T hi rows 0-7, 8-15, then lo rows 0-7, 8-15
    float alpha_a[NT], alpha_b[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float sv[2][4];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const int nv = tt ? nvalid1 : kTile;
#pragma unroll
        for (int i = 0; i < 4; ++i) sv[tt][i] = (cc[tt][0][nt][i] + cc[tt][1][nt][i]) * scale_log2;
        if (r0 >= nv) sv[tt][0] = sv[tt][1] = -INFINITY;
        if (r0 + 8 >= nv) sv[tt][2] = sv[tt][3] = -INFINITY;
      }
      if (tok0 + 2 * kTile > ctx - Q) {  // the pair reaches the queries' own positions
        const int na = col0 + nt * 8 + 2 * (lane & 3), nb = na + 1;
        const int lim_a = na < G * Q ? ctx - Q + na / G : -1;
        const int lim_b = nb < G * Q ? ctx - Q + nb / G : -1;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
          const int t0 = tok0 + 16 * tt + r0, t1 = t0 + 8;
          if (t0 > lim_a) sv[tt][0] = -INFINITY;
          if (t0 > lim_b) sv[tt][1] = -INFINITY;
          if (t1 > lim_a) sv[tt][2] = -INFINITY;
          if (t1 > lim_b) sv[tt][3] = -INFINITY;
        }
      }
      float mx_a = fmaxf(fmaxf(sv[0][0], sv[0][2]), fmaxf(sv[1][0], sv[1][2]));
      float mx_b = fmaxf(fmaxf(sv[0][1], sv[0][3]), fmaxf(sv[1][1], sv[1][3]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
        mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
      }
      const float mn_a = fmaxf(m_a[nt], mx_a), mn_b = fmaxf(m_b[nt], mx_b);
      const float base_a = (mn_a == -INFINITY) ? 0.f : mn_a;
      const float base_b = (mn_b == -INFINITY) ? 0.f : mn_b;
      alpha_a[nt] = ex2_ftz(m_a[nt] - base_a);
      alpha_b[nt] = ex2_ftz(m_b[nt] - base_b);
      m_a[nt] = mn_a;
      m_b[nt] = mn_b;
      float la = 0.f, lb = 0.f;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const float p0 = ex2_ftz(sv[tt][0] - base_a), p1 = ex2_ftz(sv[tt][1] - base_b);
        const float p2 = ex2_ftz(sv[tt][2] - base_a), p3 = ex2_ftz(sv[tt][3] - base_b);
        const uint32_t p_top = pack_bf16x2(p0, p1), p_bot = pack_bf16x2(p2, p3);
        const uint32_t r_top = pack_bf16x2(p0 - bf16_lo(p_top), p1 - bf16_hi(p_top));
        const uint32_t r_bot = pack_bf16x2(p2 - bf16_lo(p_bot), p3 - bf16_hi(p_bot));
        la += p0 + p2;
        lb += p1 + p3;
        pb[tt][nt][0] = movmatrix_trans(p_top);
        pb[tt][nt][1] = movmatrix_trans(p_bot);
        pb[tt][nt][2] = movmatrix_trans(r_top);
        pb[tt][nt][3] = movmatrix_trans(r_bot);
      }
      l_a[nt] = l_a[nt] * alpha_a[nt] + la;
      l_b[nt] = l_b[nt] * alpha_b[nt] + lb;
    }
    const int t2 = 2 * (lane & 3);
    uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
    if (nvalid1 < kTile) {
      keep_lo = (t2 < nvalid1 ? 0x0000ffffu : 0u) | (t2 + 1 < nvalid1 ? 0xffff0000u : 0u);
      keep_hi = (t2 + 8 < nvalid1 ? 0x0000ffffu : 0u) | (t2 + 9 < nvalid1 ? 0xffff0000u : 0u);
    }
    bool moved = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) moved |= (alpha_a[nt] != 1.f) || (alpha_b[nt] != 1.f);
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          acc[nt][mt][0] *= alpha_a[nt];
          acc[nt][mt][1] *= alpha_b[nt];
          acc[nt][mt][2] *= alpha_a[nt];
          acc[nt][mt][3] *= alpha_b[nt];
        }
    }
    const RowPtr<NC> vp0(v_half0, (lane & 7) + (lane >> 4) * 8, uh + ((lane >> 3) & 1), lines);
    const RowPtr<NC> vp1(v_half1, (lane & 7) + (lane >> 4) * 8, uh + ((lane >> 3) & 1), lines);
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      uint32_t v0[4], v1[4];
      ldmatrix_x4_trans(v0, vp0.at(mt));
      ldmatrix_x4_trans(v1, vp1.at(mt));
      v1[0] &= keep_lo;
      v1[1] &= keep_lo;
      v1[2] &= keep_hi;
      v1[3] &= keep_hi;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        mma_bf16_16816(acc[nt][mt], v0, pb[0][nt][0], pb[0][nt][1]);
        mma_bf16_16816(acc[nt][mt], v1, pb[1][nt][0], pb[1][nt][1]);
        mma_bf16_16816(acc[nt][mt], v0, pb[0][nt][2], pb[0][nt][3]);
        mma_bf16_16816(acc[nt][mt], v1, pb[1][nt][2], pb[1][nt][3]);
      }
    }
  }

  // Output rows are [seq][query][head]; partial rows are [query][head].
  template <bool REST = false>
  __device__ __forceinline__ void finish(const DecodeParams& p, int seq, int kv_head, int slot,
                                         int r, int lane) {
    const int G = p.group, H = p.num_heads, Q = p.num_queries;
    const int d0 = lane >> 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float la = l_a[nt], lb = l_b[nt];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        la += __shfl_xor_sync(0xffffffffu, la, o);
        lb += __shfl_xor_sync(0xffffffffu, lb, o);
      }
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = col0 + nt * 8 + 2 * (lane & 3) + half;
        if (n >= G * Q) continue;
        const int qi = n / G, g = n % G;
        const int row = qi * H + kv_head * G + g;
        const float l = half ? lb : la, m = half ? m_b[nt] : m_a[nt];
        if (!REST && slot < 0) {
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + ((size_t)seq * Q * H + row) * D;
          const float inv = l > 0.f ? 1.f / l : 0.f;  // a query with no keys gives zeros
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            out[mt * 16 + d0] = __float2bfloat16_rn(acc[nt][mt][half] * inv);
            out[mt * 16 + d0 + 8] = __float2bfloat16_rn(acc[nt][mt][2 + half] * inv);
          }
        } else {
          const bool whole = REST && slot < 0;
          const size_t base = (whole ? (size_t)seq : (size_t)r * 2 + slot) * Q * H + row;
          float* po = (whole ? p.rest_o : p.part_o) + base * D;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            po[mt * 16 + d0] = acc[nt][mt][half];
            po[mt * 16 + d0 + 8] = acc[nt][mt][2 + half];
          }
          if (d0 == 0) {
            float* pm = (whole ? p.rest_ml : p.part_ml) + base * 2;
            pm[0] = m;
            pm[1] = l;
          }
        }
      }
    }
  }
};

// FP8 pools: weights go into the f16 product times 2^kF16Up, up to 2^14 of f16's 65504.
// Relative to the largest they then keep 11 bits down to 2^-28 and vanish below
// 2^-39 (as they are, below 2^-25: 128 k tokens 2^-25 below one token's weight are
// 0.4% of the output).  The sums carry the same factor, which the stored maxima take out.
constexpr float kF16Up = 14.f;

// Consumer for an FP8 (E4M3) pool with bf16 queries and outputs.  Codes are
// widened to f16 in registers (exact) and both products run on f16 MMAs.
// Shared-memory reads use ldmatrix on 16-bit units (two codes each):
//   Q.K  - the order of head dims inside each 16-wide k-step is permuted so
//          that lane t's four consecutive codes (dims 4t..4t+3) are its k
//          pairs (2t, 2t+1) and (2t+8, 2t+9); the query fragment is loaded in
//          the same order, so the sum is unchanged.
//   P.V  - ldmatrix.trans hands each lane two dims of two tokens; the MMA's
//          output rows are permuted so that lane l/4 owns dims 2*(l/4) and
//          +1 of each 16-wide slice, and one byte permute per register builds
//          the (token, token) pairs the A operand needs.
// Scores carry k_scale in scale_log2; v_scale is applied to the output.  The
// bf16 query converts to f16 exactly for |q| in f16's normal range
// [2^-14, 65504]; P enters as f16.
// MQ: several query tokens per sequence with a causal mask, as in
// MmaConsumerMQ: column n = col0 + (lane / 4) holds (query n / G, head n % G),
// query qi sits at position ctx - Q + qi and sees tokens up to it.
// MOD (with MQ): modified scores, as in MmaConsumerMQ.
// I8: int8 pools, whose tokens have scales of their own.  Codes widen to f16 (exact), K's scale
// multiplies the token's scores and V's its weights in fp32.  f16 does not hold any
// weight times any scale, so the scales go in as fractions of `unit`, a power of two that
// no scale so far exceeds; the accumulators count in it and follow it when it grows.
template <int D, bool MQ = false, bool MOD = false, bool I8 = false>
struct MmaConsumerF8 {
  static constexpr int KS = D / 16;
  uint32_t qb[KS][2];
  float acc[KS][4];
  float m_a, m_b, l_a, l_b;
  uint32_t lane_off = 0;  // this lane's ldmatrix row address within a half-stage (K and V alike)
  int col0 = 0;           // MQ: first (query, head) column of this warp
  ModCols mc;             // MOD
  float unit = 0.f, per_unit = 0.f;  // I8: the unit and its reciprocal
  const float* scales = nullptr;     // I8: this head's 16 K scales of a stage; V's are `v_scales_at` behind
  int v_scales_at = 0;

  __device__ __forceinline__ static void widen(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    if constexpr (I8)
      s8x4_to_f16x2x2(codes, lo, hi);
    else
      e4m3x4_to_f16x2x2(codes, lo, hi);
  }
  // I8: a token's V scale in units (0: the token is not there).
  __device__ __forceinline__ void take_unit(float most) {
    if (__any_sync(0xffffffffu, most > unit)) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      // The next power of two (at most 2^127, whose reciprocal is a normal number's; scales
      // reach 2^128 / 127).
      const float next = __uint_as_float((__float_as_uint(most) + 0x007fffffu) & 0x7f800000u);
      const float f = unit * (1.f / next);  // a power of two, or zero where it does not matter any more
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][i] *= f;
      unit = next;
      per_unit = 1.f / next;
    }
  }

  // Once per kernel: uh is the head's first 16-byte unit in the group's row.
  __device__ __forceinline__ void setup(uint32_t lines, int uh, int lane) {
    lane_off = RowPtr<1>(0u, (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), lines).a[0];
  }

  // w: KV head within the CTA's group.  MQ also takes Q, Hg and this warp's
  // first column.
  __device__ __forceinline__ void begin_segment(const unsigned char* qslot, int w, int G, int lane,
                                                int Q = 1, int Hg = 1, int col_base = 0) {
    const int t4 = 4 * (lane & 3);
    const __nv_bfloat16* qh;
    bool real;
    if constexpr (MQ) {
      col0 = col_base;
      const int n = col_base + (lane >> 2);
      real = n < G * Q;
      const int qi = real ? n / G : 0, g = real ? n % G : 0;
      qh = reinterpret_cast<const __nv_bfloat16*>(qslot) + ((size_t)qi * Hg * G + w * G + g) * D;
    } else {
      const int n = lane >> 2;
      real = n < G;
      qh = reinterpret_cast<const __nv_bfloat16*>(qslot) + (size_t)(w * G + n) * D;
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if (real) {
        const uint2 v = *reinterpret_cast<const uint2*>(qh + ks * 16 + t4);  // dims t4 .. t4+3
        qb[ks][0] = pack_f16x2(bf16_lo(v.x), bf16_hi(v.x));  // k pair (2t, 2t+1)
        qb[ks][1] = pack_f16x2(bf16_lo(v.y), bf16_hi(v.y));  // k pair (2t+8, 2t+9)
      } else {
        qb[ks][0] = 0u;
        qb[ks][1] = 0u;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[ks][i] = 0.f;
    }
    m_a = m_b = -INFINITY;
    l_a = l_b = 0.f;
    if constexpr (I8) {
      unit = 0x1p-126f;  // (so that its reciprocal is finite, too)
      per_unit = 0x1p126f;
    }
  }

  // After a segment's finish (and merge) every state register is rewritten
  // by the next begin_segment before it is read; writing them here tells the
  // compiler so, which frees them for the merge.
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      qb[ks][0] = qb[ks][1] = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[ks][i] = 0.f;
    }
    m_a = m_b = l_a = l_b = 0.f;
  }

  // MQ: tok0 (first token of the tile), ctx, G and Q give the causal limits.
  __device__ __forceinline__ void tile(uint32_t k_half, uint32_t v_half, int nvalid, float scale_log2,
                                       int lane, int tok0 = 0, int ctx = 0, int G = 1, int Q = 1,
                                       const DecodeParams* mod = nullptr, const ModTile& mo = ModTile()) {
    // Matrices of one ldmatrix.x4: (rows 0-7, bytes 0-15), (rows 8-15, 0-15),
    // (rows 0-7, 16-31), (rows 8-15, 16-31) - two k-steps / m-tiles of 16 dims.
    // Half-stages are 1 KiB aligned, so adding the lane offset keeps the
    // swizzled unit bits that at(j)'s XOR steps through.
    const uint32_t ka = k_half + lane_off, va = v_half + lane_off;
    uint32_t kr[KS / 2][4], vr[KS / 2][4];
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) ldmatrix_x4(kr[j], ka ^ ((uint32_t)(j & 3) << 5));
#pragma unroll
    for (int j = 0; j < KS / 2; ++j) ldmatrix_x4_trans(vr[j], va ^ ((uint32_t)(j & 3) << 5));

    // Scores accumulate in four independent chains (k-step mod 4).
    constexpr int NCH = KS < 4 ? KS : 4;
    float cc[NCH][4];
#pragma unroll
    for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
      for (int i = 0; i < 4; ++i) cc[ch][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      const uint32_t top = kr[ks >> 1][2 * (ks & 1)], bot = kr[ks >> 1][2 * (ks & 1) + 1];
      uint32_t a[4];
      widen(top, a[0], a[2]);  // token row g: codes 0,1 | codes 2,3
      widen(bot, a[1], a[3]);  // token row g+8
      mma_f16_16816(cc[ks % NCH], a, qb[ks][0], qb[ks][1]);
    }
#pragma unroll
    for (int ch = 1; ch < NCH; ++ch)
#pragma unroll
      for (int i = 0; i < 4; ++i) cc[0][i] += cc[ch][i];
    const int g = lane >> 2, t2 = 2 * (lane & 3);
    float s0 = cc[0][0], s1 = cc[0][1], s2 = cc[0][2], s3 = cc[0][3];
    if constexpr (MOD) {
      mod_scores(*mod, mc, mo, g, s0, s1, s2, s3);
    } else {
      float f0 = scale_log2, f1 = scale_log2;
      if constexpr (I8) {
        f0 *= scales[g];
        f1 *= scales[g + 8];
      }
      s0 *= f0;
      s1 *= f0;
      s2 *= f1;
      s3 *= f1;
      if (g >= nvalid) s0 = s1 = -INFINITY;
      if (g + 8 >= nvalid) s2 = s3 = -INFINITY;
    }
    if (MQ && !MOD && tok0 + kTile > ctx - Q) {  // only tiles reaching the queries' own positions
      // Last visible position of each column's query (-1: padding column).
      const int na = col0 + t2, nb = na + 1;
      const int lim_a = na < G * Q ? ctx - Q + na / G : -1;
      const int lim_b = nb < G * Q ? ctx - Q + nb / G : -1;
      const int t0 = tok0 + g, t1 = t0 + 8;
      if (t0 > lim_a) s0 = -INFINITY;
      if (t0 > lim_b) s1 = -INFINITY;
      if (t1 > lim_a) s2 = -INFINITY;
      if (t1 > lim_b) s3 = -INFINITY;
    }
    float mx_a = fmaxf(s0, s2), mx_b = fmaxf(s1, s3);
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
    }
    const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
    const float base_a = (mn_a == -INFINITY) ? 0.f : mn_a;
    const float base_b = (mn_b == -INFINITY) ? 0.f : mn_b;
    const float alpha_a = ex2_ftz(m_a - base_a), alpha_b = ex2_ftz(m_b - base_b);
    const float up_a = base_a - kF16Up, up_b = base_b - kF16Up;
    m_a = mn_a;
    m_b = mn_b;
    const float p0 = ex2_ftz(s0 - up_a), p1 = ex2_ftz(s1 - up_b);
    const float p2 = ex2_ftz(s2 - up_a), p3 = ex2_ftz(s3 - up_b);
    // Weights enter the f16 MMA rounded to f16 (relative error <= 2^-11,
    // half an ulp of the 10-bit fraction; kF16Up), well inside the bf16 output's
    // own rounding; the running sum keeps them in fp32.
    float w0 = p0, w1 = p1, w2 = p2, w3 = p3;
    if constexpr (I8) {
      const float v0 = g < nvalid ? scales[v_scales_at + g] : 0.f, v1 = g + 8 < nvalid ? scales[v_scales_at + g + 8] : 0.f;
      take_unit(fmaxf(v0, v1));
      const float u0 = v0 * per_unit, u1 = v1 * per_unit;
      // (A token that a query does not see has no weight, whatever its scale.)
      w0 = MQ && s0 == -INFINITY ? 0.f : p0 * u0;
      w1 = MQ && s1 == -INFINITY ? 0.f : p1 * u0;
      w2 = MQ && s2 == -INFINITY ? 0.f : p2 * u1;
      w3 = MQ && s3 == -INFINITY ? 0.f : p3 * u1;
    }
    const uint32_t p_top = pack_f16x2(w0, w1), p_bot = pack_f16x2(w2, w3);
    l_a = l_a * alpha_a + p0 + p2;
    l_b = l_b * alpha_b + p1 + p3;
    const uint32_t pb0 = movmatrix_trans(p_top), pb1 = movmatrix_trans(p_bot);
    // Each V register holds bytes (tok 2t: dim 2g, 2g+1 | tok 2t+1: dim 2g, 2g+1);
    // on the last tile of a segment, tokens past the end are zeroed (code 0
    // is +0.0) before they meet a weight.
    if (MOD ? mo.vis != 0xffffu : nvalid < kTile) {
      const uint32_t keep_lo = MOD ? keep_pair(mo.vis, t2)
                                   : (t2 < nvalid ? 0x0000ffffu : 0u) | (t2 + 1 < nvalid ? 0xffff0000u : 0u);
      const uint32_t keep_hi = MOD ? keep_pair(mo.vis, t2 + 8)
                                   : (t2 + 8 < nvalid ? 0x0000ffffu : 0u) | (t2 + 9 < nvalid ? 0xffff0000u : 0u);
#pragma unroll
      for (int j = 0; j < KS / 2; ++j) {
        vr[j][0] &= keep_lo;
        vr[j][1] &= keep_hi;
        vr[j][2] &= keep_lo;
        vr[j][3] &= keep_hi;
      }
    }
    // Once the running maxima settle, most tiles leave every alpha at 1:
    // skip the rescale then (this consumer is issue-bound).
    if (__any_sync(0xffffffffu, alpha_a != 1.f || alpha_b != 1.f)) {
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        acc[mt][0] *= alpha_a;
        acc[mt][1] *= alpha_b;
        acc[mt][2] *= alpha_a;
        acc[mt][3] *= alpha_b;
      }
    }
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      const uint32_t top = vr[mt >> 1][2 * (mt & 1)];      // tokens 2t, 2t+1
      const uint32_t bot = vr[mt >> 1][2 * (mt & 1) + 1];  // tokens 2t+8, 2t+9
      // One byte permute per register: (dim 2g: tokens 2t, 2t+1 | dim 2g+1: same).
      uint32_t a[4];
      widen(__byte_perm(top, 0u, 0x3120), a[0], a[1]);
      widen(__byte_perm(bot, 0u, 0x3120), a[2], a[3]);
      mma_f16_16816(acc[mt], a, pb0, pb1);
    }
  }

  // Two consecutive tiles of one segment in one pass: the first full (16
  // tokens from tok0), the second holding nvalid1 tokens from tok0 + 16.  Their
  // score MMAs interleave in four independent chains and one softmax update
  // covers all 32 tokens, so the fixed-latency steps (score reductions,
  // exponentials, rescale) run once per pair.
  __device__ __forceinline__ void tile2(uint32_t k_half0, uint32_t v_half0, uint32_t k_half1, uint32_t v_half1,
                                        int nvalid1, float scale_log2, int lane, int tok0 = 0, int ctx = 0,
                                        int G = 1, int Q = 1, const DecodeParams* mod = nullptr,
                                        const ModTile& mo0 = ModTile(), const ModTile& mo1 = ModTile(),
                                        const float* scales1 = nullptr) {
    const uint32_t ka[2] = {k_half0 + lane_off, k_half1 + lane_off};
    const uint32_t va[2] = {v_half0 + lane_off, v_half1 + lane_off};
    uint32_t kr[2][KS / 2][4];
#pragma unroll
    for (int j = 0; j < KS / 2; ++j)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) ldmatrix_x4(kr[tt][j], ka[tt] ^ ((uint32_t)(j & 3) << 5));
    float cc[2][2][4];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int ch = 0; ch < 2; ++ch)
#pragma unroll
        for (int i = 0; i < 4; ++i) cc[tt][ch][i] = 0.f;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const uint32_t top = kr[tt][ks >> 1][2 * (ks & 1)], bot = kr[tt][ks >> 1][2 * (ks & 1) + 1];
        uint32_t a[4];
        widen(top, a[0], a[2]);
        widen(bot, a[1], a[3]);
        mma_f16_16816(cc[tt][ks & 1], a, qb[ks][0], qb[ks][1]);
      }
    uint32_t vr[2][KS / 2][4];
#pragma unroll
    for (int j = 0; j < KS / 2; ++j)
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) ldmatrix_x4_trans(vr[tt][j], va[tt] ^ ((uint32_t)(j & 3) << 5));
    const int g = lane >> 2, t2 = 2 * (lane & 3);
    float sc[2][4];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[tt][i] = cc[tt][0][i] + cc[tt][1][i];
        if constexpr (!MOD) {
          float f = scale_log2;
          if constexpr (I8) f *= (tt ? scales1 : scales)[g + 8 * (i >> 1)];
          sc[tt][i] *= f;
        }
      }
    if constexpr (MOD) {
      mod_scores(*mod, mc, mo0, g, sc[0][0], sc[0][1], sc[0][2], sc[0][3]);
      mod_scores(*mod, mc, mo1, g, sc[1][0], sc[1][1], sc[1][2], sc[1][3]);
    } else {
      if (g >= nvalid1) sc[1][0] = sc[1][1] = -INFINITY;
      if (g + 8 >= nvalid1) sc[1][2] = sc[1][3] = -INFINITY;
    }
    if (MQ && !MOD && tok0 + 2 * kTile > ctx - Q) {  // the pair reaches the queries' own positions
      const int na = col0 + t2, nb = na + 1;
      const int lim_a = na < G * Q ? ctx - Q + na / G : -1;
      const int lim_b = nb < G * Q ? ctx - Q + nb / G : -1;
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const int t0 = tok0 + 16 * tt + g, t1 = t0 + 8;
        if (t0 > lim_a) sc[tt][0] = -INFINITY;
        if (t0 > lim_b) sc[tt][1] = -INFINITY;
        if (t1 > lim_a) sc[tt][2] = -INFINITY;
        if (t1 > lim_b) sc[tt][3] = -INFINITY;
      }
    }
    float mx_a = fmaxf(fmaxf(sc[0][0], sc[0][2]), fmaxf(sc[1][0], sc[1][2]));
    float mx_b = fmaxf(fmaxf(sc[0][1], sc[0][3]), fmaxf(sc[1][1], sc[1][3]));
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      mx_a = fmaxf(mx_a, __shfl_xor_sync(0xffffffffu, mx_a, o));
      mx_b = fmaxf(mx_b, __shfl_xor_sync(0xffffffffu, mx_b, o));
    }
    const float mn_a = fmaxf(m_a, mx_a), mn_b = fmaxf(m_b, mx_b);
    const float base_a = (mn_a == -INFINITY) ? 0.f : mn_a;
    const float base_b = (mn_b == -INFINITY) ? 0.f : mn_b;
    const float alpha_a = ex2_ftz(m_a - base_a), alpha_b = ex2_ftz(m_b - base_b);
    const float up_a = base_a - kF16Up, up_b = base_b - kF16Up;
    m_a = mn_a;
    m_b = mn_b;
    float pw[2][4];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
      pw[tt][0] = ex2_ftz(sc[tt][0] - up_a);
      pw[tt][1] = ex2_ftz(sc[tt][1] - up_b);
      pw[tt][2] = ex2_ftz(sc[tt][2] - up_a);
      pw[tt][3] = ex2_ftz(sc[tt][3] - up_b);
    }
    l_a = l_a * alpha_a + ((pw[0][0] + pw[0][2]) + (pw[1][0] + pw[1][2]));
    l_b = l_b * alpha_b + ((pw[0][1] + pw[0][3]) + (pw[1][1] + pw[1][3]));
    if constexpr (I8) {
      float u[2][2];
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          u[tt][i] = tt == 0 || g + 8 * i < nvalid1 ? (tt ? scales1 : scales)[v_scales_at + g + 8 * i] : 0.f;
      take_unit(fmaxf(fmaxf(u[0][0], u[0][1]), fmaxf(u[1][0], u[1][1])));
#pragma unroll
      for (int tt = 0; tt < 2; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          pw[tt][i] = MQ && sc[tt][i] == -INFINITY ? 0.f : pw[tt][i] * (u[tt][i >> 1] * per_unit);
    }
    uint32_t pb[2][2];
#pragma unroll
    for (int tt = 0; tt < 2; ++tt) {
      pb[tt][0] = movmatrix_trans(pack_f16x2(pw[tt][0], pw[tt][1]));
      pb[tt][1] = movmatrix_trans(pack_f16x2(pw[tt][2], pw[tt][3]));
    }
    if constexpr (MOD) {
#pragma unroll
      for (int tt = 0; tt < 2; ++tt) {
        const uint32_t vis = tt ? mo1.vis : mo0.vis;
        if (vis != 0xffffu) {
          const uint32_t keep_lo = keep_pair(vis, t2), keep_hi = keep_pair(vis, t2 + 8);
#pragma unroll
          for (int j = 0; j < KS / 2; ++j) {
            vr[tt][j][0] &= keep_lo;
            vr[tt][j][1] &= keep_hi;
            vr[tt][j][2] &= keep_lo;
            vr[tt][j][3] &= keep_hi;
          }
        }
      }
    } else if (nvalid1 < kTile) {
      const uint32_t keep_lo = (t2 < nvalid1 ? 0x0000ffffu : 0u) | (t2 + 1 < nvalid1 ? 0xffff0000u : 0u);
      const uint32_t keep_hi = (t2 + 8 < nvalid1 ? 0x0000ffffu : 0u) | (t2 + 9 < nvalid1 ? 0xffff0000u : 0u);
#pragma unroll
      for (int j = 0; j < KS / 2; ++j) {
        vr[1][j][0] &= keep_lo;
        vr[1][j][1] &= keep_hi;
        vr[1][j][2] &= keep_lo;
        vr[1][j][3] &= keep_hi;
      }
    }
    if (__any_sync(0xffffffffu, alpha_a != 1.f || alpha_b != 1.f)) {
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        acc[mt][0] *= alpha_a;
        acc[mt][1] *= alpha_b;
        acc[mt][2] *= alpha_a;
        acc[mt][3] *= alpha_b;
      }
    }
#pragma unroll
    for (int tt = 0; tt < 2; ++tt)
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        const uint32_t top = vr[tt][mt >> 1][2 * (mt & 1)];
        const uint32_t bot = vr[tt][mt >> 1][2 * (mt & 1) + 1];
        uint32_t a[4];
        widen(__byte_perm(top, 0u, 0x3120), a[0], a[1]);
        widen(__byte_perm(bot, 0u, 0x3120), a[2], a[3]);
        mma_f16_16816(acc[mt], a, pb[tt][0], pb[tt][1]);
      }
  }

  // Output row pairs: acc[mt][0] / [2] are dims dd / dd+1 of column a,
  // [1] / [3] of column b.  Output rows are [seq][query][head]; partial rows
  // are [query][head] (one query: [head]).
  template <bool REST = false>
  __device__ __forceinline__ void finish(const DecodeParams& p, int seq, int kv_head, int slot,
                                         int r, int lane) {
    float la = l_a, lb = l_b;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      la += __shfl_xor_sync(0xffffffffu, la, o);
      lb += __shfl_xor_sync(0xffffffffu, lb, o);
    }
    const int G = p.group, H = p.num_heads, Q = MQ ? p.num_queries : 1;
    const int g = lane >> 2;
    const float v_scale = I8 ? 1.f : p.v_scale;
    if constexpr (I8) {
      // The unit may be near the largest number and the weights count 2^14 times: with both a row's
      // sums and those of its weights 2^14 times smaller (here and in every other partial) a row
      // stays finite as long as the sum of its weights of at most 1 times |v| does, as over other pools.
      constexpr float kDown = 0x1p-14f;
      static_assert(kF16Up == 14.f, "the weights' factor");
      const float by = unit * kDown;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[mt][i] *= by;
      la *= kDown;
      lb *= kDown;
    }
    if constexpr (!MQ) {
      const int ha = 2 * (lane & 3), hb = ha + 1;
      const int qa = kv_head * G + ha, qb_ = kv_head * G + hb;
      if (slot < 0) {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + (size_t)seq * H * D;
        const float ia = v_scale / la, ib = v_scale / lb;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int dd = mt * 16 + 2 * g;
          if (ha < G)
            *reinterpret_cast<uint32_t*>(out + (size_t)qa * D + dd) = pack_bf16x2(acc[mt][0] * ia, acc[mt][2] * ia);
          if (hb < G)
            *reinterpret_cast<uint32_t*>(out + (size_t)qb_ * D + dd) = pack_bf16x2(acc[mt][1] * ib, acc[mt][3] * ib);
        }
      } else {
        const size_t base = ((size_t)r * 2 + slot) * H;
        float* po = p.part_o + base * D;
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          const int dd = mt * 16 + 2 * g;
          if (ha < G) *reinterpret_cast<float2*>(po + (size_t)qa * D + dd) = make_float2(acc[mt][0], acc[mt][2]);
          if (hb < G) *reinterpret_cast<float2*>(po + (size_t)qb_ * D + dd) = make_float2(acc[mt][1], acc[mt][3]);
        }
        if (g == 0) {
          float* pm = p.part_ml + base * 2;
          if (ha < G) *reinterpret_cast<float2*>(pm + (size_t)qa * 2) = make_float2(m_a - kF16Up, la);
          if (hb < G) *reinterpret_cast<float2*>(pm + (size_t)qb_ * 2) = make_float2(m_b - kF16Up, lb);
        }
      }
    } else {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int n = col0 + 2 * (lane & 3) + half;
        if (n >= G * Q) continue;
        int qi = 0, gh = n;
        if constexpr (MQ) {
          qi = n / G;
          gh = n % G;
        }
        const int row = qi * H + kv_head * G + gh;
        const float l = half ? lb : la, m = (half ? m_b : m_a) - kF16Up;
        if (!REST && slot < 0) {
          __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + ((size_t)seq * Q * H + row) * D;
          // A query with no keys (several queries, short context) gives zeros.
          const float inv = (!MQ || (I8 ? l != 0.f : l > 0.f)) ? v_scale / l : 0.f;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt)
            *reinterpret_cast<uint32_t*>(out + mt * 16 + 2 * g) =
                pack_bf16x2(acc[mt][half] * inv, acc[mt][2 + half] * inv);
        } else {
          const bool whole = REST && slot < 0;
          const size_t base = (whole ? (size_t)seq : (size_t)r * 2 + slot) * Q * H + row;
          float* po = (whole ? p.rest_o : p.part_o) + base * D;
#pragma unroll
          for (int mt = 0; mt < KS; ++mt)
            *reinterpret_cast<float2*>(po + mt * 16 + 2 * g) = make_float2(acc[mt][half], acc[mt][2 + half]);
          if (g == 0)
            *reinterpret_cast<float2*>((whole ? p.rest_ml : p.part_ml) + base * 2) = make_float2(m, l);
        }
      }
    }
  }
};

// Consumer for more than 8 (query, head) columns per KV head in the walks other
// than kWalkAll: 16 of them per warp, as the rows of the products.  S[16 x tokens] =
// Q K^T with Q as the A operand, and the weights are A again for O[16 x D] += P V
// straight from the score registers.  Against 8 columns per warp (S^T = K Q^T) it
// reads, and for FP8 pools widens, every K and V fragment once for 16 rows, needs
// two shuffles per reduction instead of three and no transpose of P: 48 sequences x
// 4 queries over FP8 pools 75 -> 57 us, 96 x 3 over 64 dims 99 -> 66.  What bounds it is
// instruction issue and its latencies (10 to 15 warps per SM, 35 to 46% of issue
// slots); one tile a pass gives 98 and 74 us, four 85 and 110 (registers spill).
//   bf16: P as a high and a low bf16 part (about 2^-16).  FP8 pools: codes widened
//   to f16, head dims inside a 16-wide k-step in the order 4t .. 4t + 3 per lane
//   (see MmaConsumerF8), P rounded to f16.
// Lane l holds rows l / 4 and l / 4 + 8 and, of a tile's scores, tokens 2 (l % 4),
// + 1, + 8, + 9.
template <int D, bool KV8, bool MOD>
struct RowsConsumer {
  static constexpr int KS = D / 16;
  static constexpr int NC = D * 2 > 128 ? D * 2 / 128 : 1;
  uint32_t qf[KS][4];
  float acc[D / 8][4];  // KV8: tiles 2j and 2j + 1 are the even and odd dims of slice j
  float m[2], l[2];
  int row0 = 0;
  uint32_t lane_off = 0;  // KV8: this lane's ldmatrix row address within a half-stage
  ModCols mc;             // rows l / 4 and l / 4 + 8

  __device__ __forceinline__ void setup(const DecodeParams& p, int kv_head, int first_row, int w, int lane) {
    row0 = first_row;
    const int G = p.group, n = G * p.num_queries, a = row0 + (lane >> 2), b = a + 8;
    mc.qa = a < n ? a / G : 0;
    mc.qb = b < n ? b / G : 0;
    if (MOD && p.slopes != nullptr) {
      if (a < n) mc.sa = 1.4426950408889634f * __ldg(p.slopes + kv_head * G + a % G);
      if (b < n) mc.sb = 1.4426950408889634f * __ldg(p.slopes + kv_head * G + b % G);
    }
    if constexpr (KV8)
      lane_off = RowPtr<1>(0u, (lane & 7) + ((lane >> 3) & 1) * 8, w * D / 16 + (lane >> 4), p.lines).a[0];
  }

  __device__ __forceinline__ void begin_segment(const DecodeParams& p, const unsigned char* qslot, int w, int lane) {
    const int G = p.group, n = G * p.num_queries, Hg = p.heads_per_cta, t = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = row0 + (lane >> 2) + 8 * half;
      const bool real = r < n;
      const int qi = real ? r / G : 0, g = real ? r % G : 0;
      const __nv_bfloat16* q =
          reinterpret_cast<const __nv_bfloat16*>(qslot) + ((size_t)qi * Hg * G + w * G + g) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (KV8) {
          const uint2 v = real ? *reinterpret_cast<const uint2*>(q + ks * 16 + 4 * t) : make_uint2(0u, 0u);
          qf[ks][half] = pack_f16x2(bf16_lo(v.x), bf16_hi(v.x));
          qf[ks][2 + half] = pack_f16x2(bf16_lo(v.y), bf16_hi(v.y));
        } else {
          qf[ks][half] = real ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 2 * t) : 0u;
          qf[ks][2 + half] = real ? *reinterpret_cast<const uint32_t*>(q + ks * 16 + 8 + 2 * t) : 0u;
        }
      }
      m[half] = -INFINITY;
      l[half] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  }

  // N tiles (1 or 2) of one segment in one pass.
  template <int N>
  __device__ __forceinline__ void tiles(const DecodeParams& p, const uint32_t (&kh)[N], const uint32_t (&vh)[N], int uh,
                                        const ModTile (&mo)[N], int lane) {
    const int t2 = 2 * (lane & 3);
    // Scores: the tiles' chains interleave (k-steps outside), two per tile.
    float s[N][8], c[N][2][4];  // c: tokens 0-7, 8-15
#pragma unroll
    for (int tt = 0; tt < N; ++tt)
#pragma unroll
      for (int i = 0; i < 4; ++i) c[tt][0][i] = c[tt][1][i] = 0.f;
    if constexpr (KV8) {
#pragma unroll
      for (int j = 0; j < KS / 2; ++j) {
        uint32_t kr[N][4];
#pragma unroll
        for (int tt = 0; tt < N; ++tt) ldmatrix_x4(kr[tt], (kh[tt] + lane_off) ^ ((uint32_t)(j & 3) << 5));
#pragma unroll
        for (int i = 0; i < 4; ++i)  // k-step 2j + i / 2, tokens 8 (i % 2) ..
#pragma unroll
          for (int tt = 0; tt < N; ++tt) {
            uint32_t b0, b1;
            e4m3x4_to_f16x2x2(kr[tt][i], b0, b1);
            mma_f16_16816(c[tt][i & 1], qf[2 * j + (i >> 1)], b0, b1);
          }
      }
    } else {
      uint32_t ka[N][NC];
#pragma unroll
      for (int tt = 0; tt < N; ++tt) {
        const RowPtr<NC> kp(kh[tt], (lane & 7) + ((lane >> 4) & 1) * 8, uh + ((lane >> 3) & 1), p.lines);
#pragma unroll
        for (int i = 0; i < NC; ++i) ka[tt][i] = kp.a[i];
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int tt = 0; tt < N; ++tt) {
          uint32_t b[4];
          ldmatrix_x4(b, ka[tt][ks >> 2] ^ ((uint32_t)(ks & 3) << 5));
          mma_bf16_16816(c[tt][0], qf[ks], b[0], b[1]);
          mma_bf16_16816(c[tt][1], qf[ks], b[2], b[3]);
        }
    }
#pragma unroll
    for (int tt = 0; tt < N; ++tt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s[tt][2 * i] = c[tt][i][0], s[tt][2 * i + 1] = c[tt][i][1];
        s[tt][4 + 2 * i] = c[tt][i][2], s[tt][5 + 2 * i] = c[tt][i][3];
      }
      row_scores<MOD>(p, mc, mo[tt], t2, s[tt]);
    }
    float alpha[2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float mx = s[0][4 * half];
#pragma unroll
      for (int tt = 0; tt < N; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[tt][4 * half + i]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[half], mx);
      // A row may see no token of these tiles (or none yet): keep -inf out of the exponent base.
      const float base = mn == -INFINITY ? 0.f : mn;
      alpha[half] = ex2_ftz(m[half] - base);
      m[half] = mn;
      const float up = KV8 ? base - kF16Up : base;
      float sum = 0.f;
#pragma unroll
      for (int tt = 0; tt < N; ++tt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[tt][4 * half + i] = ex2_ftz(s[tt][4 * half + i] - up);
          sum += s[tt][4 * half + i];
        }
      l[half] = l[half] * alpha[half] + sum;
    }
    // Rescale the accumulators only when some running maximum moved.
    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        acc[i][0] *= alpha[0];
        acc[i][1] *= alpha[0];
        acc[i][2] *= alpha[1];
        acc[i][3] *= alpha[1];
      }
    }
#pragma unroll
    for (int tt = 0; tt < N; ++tt) {
      const float (&w)[8] = s[tt];
      uint32_t keep_lo = 0xffffffffu, keep_hi = 0xffffffffu;
      if (mo[tt].vis != 0xffffu) {
        // V entries of rows nobody sees may be non-finite: zero them.
        keep_lo = keep_pair(mo[tt].vis, t2);
        keep_hi = keep_pair(mo[tt].vis, t2 + 8);
      }
      if constexpr (KV8) {
        const uint32_t a[4] = {pack_f16x2(w[0], w[1]), pack_f16x2(w[4], w[5]), pack_f16x2(w[2], w[3]),
                               pack_f16x2(w[6], w[7])};
        const uint32_t va = vh[tt] + lane_off;
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
          uint32_t vr[4];
          ldmatrix_x4_trans(vr, va ^ ((uint32_t)(j & 3) << 5));
#pragma unroll
          for (int i = 0; i < 2; ++i) {  // slice 2j + i
            uint32_t e0, o0, e1, o1;     // even and odd dims, tokens 0-7 and 8-15
            e4m3x4_to_f16x2x2(__byte_perm(vr[2 * i] & keep_lo, 0u, 0x3120), e0, o0);
            e4m3x4_to_f16x2x2(__byte_perm(vr[2 * i + 1] & keep_hi, 0u, 0x3120), e1, o1);
            mma_f16_16816(acc[2 * (2 * j + i)], a, e0, e1);
            mma_f16_16816(acc[2 * (2 * j + i) + 1], a, o0, o1);
          }
        }
      } else {
        const uint32_t a[4] = {pack_bf16x2(w[0], w[1]), pack_bf16x2(w[4], w[5]), pack_bf16x2(w[2], w[3]),
                               pack_bf16x2(w[6], w[7])};
        const uint32_t r[4] = {pack_bf16x2(w[0] - bf16_lo(a[0]), w[1] - bf16_hi(a[0])),
                               pack_bf16x2(w[4] - bf16_lo(a[1]), w[5] - bf16_hi(a[1])),
                               pack_bf16x2(w[2] - bf16_lo(a[2]), w[3] - bf16_hi(a[2])),
                               pack_bf16x2(w[6] - bf16_lo(a[3]), w[7] - bf16_hi(a[3]))};
        const RowPtr<NC> vp(vh[tt], (lane & 7) + ((lane >> 3) & 1) * 8, uh + (lane >> 4), p.lines);
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          uint32_t b[4];
          ldmatrix_x4_trans(b, vp.at(mt));
          b[0] &= keep_lo;
          b[1] &= keep_hi;
          b[2] &= keep_lo;
          b[3] &= keep_hi;
          mma_bf16_16816(acc[2 * mt], a, b[0], b[1]);
          mma_bf16_16816(acc[2 * mt + 1], a, b[2], b[3]);
          mma_bf16_16816(acc[2 * mt], r, b[0], b[1]);
          mma_bf16_16816(acc[2 * mt + 1], r, b[2], b[3]);
        }
      }
    }
  }

  // slot < 0: final output (REST: the row's (m, l, O)); else partial slot of range r.
  template <bool REST = false>
  __device__ __forceinline__ void finish(const DecodeParams& p, int seq, int kv_head, int slot, int r, int lane) {
    const int G = p.group, H = p.num_heads, Q = p.num_queries, t = lane & 3;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      float sum = l[half];
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      const int n = row0 + (lane >> 2) + 8 * half;
      if (n >= G * Q) continue;
      const int row = (n / G) * H + kv_head * G + n % G;
      const bool whole = slot < 0;
      if (!REST && whole) {
        __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(p.out) + ((size_t)seq * Q * H + row) * D;
        const float inv = sum > 0.f ? p.v_scale / sum : 0.f;  // a query that sees nothing gives zeros
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float (&a)[4] = acc[2 * j], (&b)[4] = acc[2 * j + 1];
          if constexpr (KV8) {
            *reinterpret_cast<uint2*>(out + 16 * j + 4 * t) =
                make_uint2(pack_bf16x2(a[2 * half] * inv, b[2 * half] * inv),
                           pack_bf16x2(a[2 * half + 1] * inv, b[2 * half + 1] * inv));
          } else {
            *reinterpret_cast<uint32_t*>(out + 16 * j + 2 * t) = pack_bf16x2(a[2 * half] * inv, a[2 * half + 1] * inv);
            *reinterpret_cast<uint32_t*>(out + 16 * j + 8 + 2 * t) =
                pack_bf16x2(b[2 * half] * inv, b[2 * half + 1] * inv);
          }
        }
      } else {
        const size_t at = (whole ? (size_t)seq : (size_t)r * 2 + slot) * Q * H + row;
        float* po = (whole ? p.rest_o : p.part_o) + at * D;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float (&a)[4] = acc[2 * j], (&b)[4] = acc[2 * j + 1];
          if constexpr (KV8) {
            *reinterpret_cast<float4*>(po + 16 * j + 4 * t) =
                make_float4(a[2 * half], b[2 * half], a[2 * half + 1], b[2 * half + 1]);
          } else {
            *reinterpret_cast<float2*>(po + 16 * j + 2 * t) = make_float2(a[2 * half], a[2 * half + 1]);
            *reinterpret_cast<float2*>(po + 16 * j + 8 + 2 * t) = make_float2(b[2 * half], b[2 * half + 1]);
          }
        }
        if (t == 0)
          *reinterpret_cast<float2*>((whole ? p.rest_ml : p.part_ml) + at * 2) = make_float2(KV8 ? m[half] - kF16Up : m[half], sum);
      }
    }
  }
};

// fp32 CUDA-core consumer.  Lane l owns head dims [l*DC, l*DC+DC) of every
// query head; after the butterfly reduction lane l holds the score of token l/2.
template <int D, int GMAX>
struct SimtConsumer {
  static constexpr int DC = D / 32;
  float qv[GMAX][DC];
  float acc[GMAX][DC];
  float m[GMAX], l[GMAX];  // l: this lane's share (token l/2, counted on even and odd lanes)

  __device__ __forceinline__ void begin_segment(const unsigned char* qslot, int w, int G,
                                                int lane) {
    const float* qh = reinterpret_cast<const float*>(qslot) + (size_t)w * G * D;
#pragma unroll
    for (int h = 0; h < GMAX; ++h) {
#pragma unroll
      for (int i = 0; i < DC; ++i) {
        qv[h][i] = (h < G) ? qh[(size_t)h * D + lane * DC + i] : 0.f;
        acc[h][i] = 0.f;
      }
      m[h] = -INFINITY;
      l[h] = 0.f;
    }
  }

  __device__ __forceinline__ void tile(const unsigned char* k_base, const unsigned char* v_base,
                                       uint32_t pitch, int nvalid, float scale_log2, int G,
                                       int lane) {
    const int my_tok = lane >> 1;
#pragma unroll
    for (int h = 0; h < GMAX; ++h) {
      if (h >= G) break;
      float part[kTile];
#pragma unroll
      for (int t = 0; t < kTile; ++t) {
        const float* kr = reinterpret_cast<const float*>(k_base + t * pitch) + lane * DC;
        float sacc = 0.f;
#pragma unroll
        for (int i = 0; i < DC; ++i) sacc = fmaf(qv[h][i], kr[i], sacc);
        part[t] = sacc;
      }
      // Butterfly reduce-scatter: 16 partial sums over 32 lanes -> one full sum
      // per lane pair.  Step xor 16 keeps the half selected by lane bit 4, etc.
      float v8[8], v4[4], v2[2];
      const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4, b1 = lane & 2;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float mine = b4 ? part[i + 8] : part[i];
        const float give = b4 ? part[i] : part[i + 8];
        v8[i] = mine + __shfl_xor_sync(0xffffffffu, give, 16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float mine = b3 ? v8[i + 4] : v8[i];
        const float give = b3 ? v8[i] : v8[i + 4];
        v4[i] = mine + __shfl_xor_sync(0xffffffffu, give, 8);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float mine = b2 ? v4[i + 2] : v4[i];
        const float give = b2 ? v4[i] : v4[i + 2];
        v2[i] = mine + __shfl_xor_sync(0xffffffffu, give, 4);
      }
      float sc;
      {
        const float mine = b1 ? v2[1] : v2[0];
        const float give = b1 ? v2[0] : v2[1];
        sc = mine + __shfl_xor_sync(0xffffffffu, give, 2);
      }
      sc += __shfl_xor_sync(0xffffffffu, sc, 1);
      sc *= scale_log2;
      if (my_tok >= nvalid) sc = -INFINITY;
      float mx = sc;
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float mn = fmaxf(m[h], mx);
      const float base = (mn == -INFINITY) ? 0.f : mn;
      const float alpha = ex2_ftz(m[h] - base);
      m[h] = mn;
      const float pw = ex2_ftz(sc - base);
      l[h] = l[h] * alpha + pw;
#pragma unroll
      for (int i = 0; i < DC; ++i) acc[h][i] *= alpha;
      for (int t = 0; t < nvalid; ++t) {
        const float pt = __shfl_sync(0xffffffffu, pw, 2 * t);
        const float* vr = reinterpret_cast<const float*>(v_base + t * pitch) + lane * DC;
#pragma unroll
        for (int i = 0; i < DC; ++i) acc[h][i] = fmaf(pt, vr[i], acc[h][i]);
      }
    }
  }

  __device__ __forceinline__ void finish(const DecodeParams& p, int seq, int kv_head, int slot,
                                         int r, int lane) {
    const int G = p.group, H = p.num_heads;
#pragma unroll
    for (int h = 0; h < GMAX; ++h) {
      if (h >= G) break;
      float lt = l[h];
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
      const int qh = kv_head * G + h;
      if (slot < 0) {
        float* out = reinterpret_cast<float*>(p.out) + ((size_t)seq * H + qh) * D + lane * DC;
        const float inv = 1.f / lt;
#pragma unroll
        for (int i = 0; i < DC; ++i) out[i] = acc[h][i] * inv;
      } else {
        const size_t base = ((size_t)r * 2 + slot) * H + qh;
        float* po = p.part_o + base * D + lane * DC;
#pragma unroll
        for (int i = 0; i < DC; ++i) po[i] = acc[h][i];
        if (lane == 0) {
          p.part_ml[base * 2 + 0] = m[h];
          p.part_ml[base * 2 + 1] = lt;
        }
      }
    }
  }
};

// fp32 consumer with modified scores (one query, at position ctx - 1).  Scores:
// lanes 2t and 2t + 1 take one half of token t's dims each, for all G heads of the
// group, so a K value is read from shared memory once; the queries are read
// there too, as broadcasts.  Of a token's finished scores the even lane keeps the
// even heads and the odd lane the odd ones: cap, bias, maximum, exponential.
// Output: lane l owns dims [l * D / 32, (l + 1) * D / 32) of all heads, the weights
// come back through a small buffer.  Products run two to an instruction.  Bound by
// shared-memory reads and products: 3 sequences of 3k to 9k tokens, 8 query heads of 128
// per KV head, 4 KV heads, 149 us with every head's K read apart, 43 us so (11 us of HBM time).
template <int D, int GMAX>
struct Fp32ModConsumer {
  static constexpr int DC = D / 32, DP = DC / 2;  // dims per lane, as pairs
  static constexpr int GH = (GMAX + 1) / 2;       // heads a lane keeps
  uint64_t acc[GMAX][DP];
  float m[GH], l[GH], slope[GH];
  const unsigned char* q;  // the segment's queries of this KV head: [G][D]

  __device__ __forceinline__ void setup(const DecodeParams& p, int kv_head, int lane) {
#pragma unroll
    for (int i = 0; i < GH; ++i) {
      const int h = 2 * i + (lane & 1);
      slope[i] = p.slopes != nullptr && h < p.group
                     ? 1.4426950408889634f * __ldg(p.slopes + kv_head * p.group + h) : 0.f;
    }
  }

  __device__ __forceinline__ void begin_segment(const unsigned char* qslot, int w, int G) {
    q = qslot + (size_t)w * G * D * 4;
#pragma unroll
    for (int h = 0; h < GMAX; ++h)
#pragma unroll
      for (int i = 0; i < DP; ++i) acc[h][i] = 0ull;
#pragma unroll
    for (int i = 0; i < GH; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
  }

  // weights: this warp's [kTile + 1][GMAX] pairs (each weight twice, then the
  // factors of the accumulators).
  __device__ __forceinline__ void tile(const DecodeParams& p, const unsigned char* k_base, const unsigned char* v_base,
                                       const ModTile& mo, float2* weights, int lane) {
    const int G = p.group, t = lane >> 1, odd = lane & 1;
    // Scores: dims [odd * D / 2, (odd + 1) * D / 2) of token t.
    uint64_t s2[GMAX];
#pragma unroll
    for (int h = 0; h < GMAX; ++h) s2[h] = 0ull;
    const unsigned char* kr = k_base + t * p.pitch + odd * (D * 2);
    const unsigned char* qr = q + odd * (D * 2);
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const int c = i ^ (4 * odd);  // the two halves in different banks
      const ulonglong2 kv = *reinterpret_cast<const ulonglong2*>(kr + 16 * c);
#pragma unroll
      for (int h = 0; h < GMAX; ++h) {
        if (h < G) {
          const ulonglong2 qv = *reinterpret_cast<const ulonglong2*>(qr + h * (D * 4) + 16 * c);
          s2[h] = fma_pair(kv.x, qv.x, s2[h]);
          s2[h] = fma_pair(kv.y, qv.y, s2[h]);
        }
      }
    }
    const bool seen = (mo.vis >> t) & 1u;
    const float dist = fabsf(static_cast<float>(mo.ctx - 1 - mo.tok0 - t));
#pragma unroll
    for (int i = 0; i < GH; ++i) {
      // This lane's half of heads 2i and 2i + 1: give the other lane its head's.
      float a, b, e = 0.f, f = 0.f;
      unpair(s2[2 * i], a, b);
      if (2 * i + 1 < GMAX) unpair(s2[2 * i + 1 < GMAX ? 2 * i + 1 : 0], e, f);
      const float even = a + b, odds = e + f;
      const float other = __shfl_xor_sync(0xffffffffu, odd ? even : odds, 1);
      float sc = (odd ? odds : even) + other;
      // fp32 outputs keep the cap's full precision: tanhf, not the SFU form.  Below
      // 2^-13 of the cap tanh(t) is t to fp32 (t^2 / 3 < 2^-27).
      const float arg = sc * p.cap_in;
      sc = p.cap_out != 0.f && fabsf(arg) >= 0x1p-13f ? p.cap_out * tanhf(arg) : sc * p.scale_log2;
      sc -= slope[i] * dist;
      if (!seen) sc = -INFINITY;
      float mx = sc;
#pragma unroll
      for (int o2 = 2; o2 < 32; o2 <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o2));
      const float mn = fmaxf(m[i], mx);
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float alpha = ex2_ftz(m[i] - ref), w = ex2_ftz(sc - ref);
      m[i] = mn;
      l[i] = l[i] * alpha + w;
      const int h = 2 * i + odd;
      if (h < GMAX) {
        weights[t * GMAX + h] = make_float2(w, w);
        if (t == 0) weights[kTile * GMAX + h] = make_float2(alpha, alpha);
      }
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < GMAX; ++h) {
      if (h < G) {
        const uint64_t f = *reinterpret_cast<const uint64_t*>(weights + kTile * GMAX + h);
#pragma unroll
        for (int i = 0; i < DP; ++i) acc[h][i] = mul_pair(acc[h][i], f);
      }
    }
#pragma unroll 4
    for (int tt = 0; tt < kTile; ++tt) {
      if (!((mo.vis >> tt) & 1u)) continue;  // its V row may be non-finite
      const unsigned char* vr = v_base + tt * p.pitch + lane * DC * 4;
      uint64_t v[DP];
      if constexpr (DP == 2) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(vr);
        v[0] = x.x, v[1] = x.y;
      } else {
        v[0] = *reinterpret_cast<const uint64_t*>(vr);
      }
#pragma unroll
      for (int h = 0; h < GMAX; ++h) {
        if (h < G) {
          const uint64_t w = *reinterpret_cast<const uint64_t*>(weights + tt * GMAX + h);
#pragma unroll
          for (int i = 0; i < DP; ++i) acc[h][i] = fma_pair(v[i], w, acc[h][i]);
        }
      }
    }
    __syncwarp();
  }

  __device__ __forceinline__ void finish(const DecodeParams& p, int seq, int kv_head, int slot, int r, int lane) {
    const int G = p.group, H = p.num_heads;
#pragma unroll
    for (int h = 0; h < GMAX; ++h) {
      float lt = l[h / 2];
#pragma unroll
      for (int o2 = 2; o2 < 32; o2 <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o2);
      lt = __shfl_sync(0xffffffffu, lt, h & 1);
      const float mt = __shfl_sync(0xffffffffu, m[h / 2], h & 1);
      if (h >= G) continue;
      const int qh = kv_head * G + h;
      const size_t base = slot < 0 ? (size_t)seq * H + qh : ((size_t)r * 2 + slot) * H + qh;
      const float f = slot < 0 ? 1.f / lt : 1.f;  // a sequence with tiles has a seen token
      float* o = (slot < 0 ? reinterpret_cast<float*>(p.out) : p.part_o) + base * D + lane * DC;
#pragma unroll
      for (int i = 0; i < DP; ++i) {
        float a, b;
        unpair(acc[h][i], a, b);
        *reinterpret_cast<float2*>(o + 2 * i) = make_float2(a * f, b * f);
      }
      if (slot >= 0 && lane == 0) *reinterpret_cast<float2*>(p.part_ml + base * 2) = make_float2(mt, lt);
    }
  }
};

// Zero the output rows of an empty sequence (16-byte stores; rows are 16-byte multiples).
template <typename T, int D>
__device__ void zero_row(const DecodeParams& p, int s) {
  // Output rows of sequence s: [num_queries][num_heads][D].
  const size_t n = (size_t)p.num_queries * p.num_heads * D;
  const size_t n16 = n * sizeof(T) / 16;
  uint4* o = reinterpret_cast<uint4*>(reinterpret_cast<T*>(p.out) + (size_t)s * n);
  for (size_t i = 0; i < n16; ++i) o[i] = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ float warp_max_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float warp_sum_f(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Called by a consumer warp right after it wrote its partial (m, l, O) for
// (seq, kv_head).  Takes a ticket; the warp holding the last of the r1-r0+1
// tickets merges every partial of that sequence and KV head by log-sum-exp,
// writes the output rows, and resets the ticket counter.  Nobody waits.
// `arrivals`: warps writing partials per range and KV head (two to four when
// the (query, head) columns of a KV head are split across several warps).
template <typename T, int D, bool kMQ>
__device__ void arrive_and_merge(const DecodeParams& p, int seq, int kv_head, int r0, int r1,
                                 int slot0, int lane, int arrivals = 1) {
  // Release: the warp barrier orders every lane's partial stores before lane
  // 0's fence, which makes them visible device-wide before the ticket.
  // Acquire: the warp holding the last ticket fences before the barrier that
  // releases its lanes to read the other partials.
  const int last = arrivals * (r1 - r0 + 1) - 1;
  int* cnt = p.counters + (size_t)r0 * p.num_kv_heads + kv_head;
  __syncwarp();
  int ticket = 0;
  if (lane == 0) {
    __threadfence();
    ticket = atomicAdd(cnt, 1);
    if (ticket == last) __threadfence();
  }
  __syncwarp();
  ticket = __shfl_sync(0xffffffffu, ticket, 0);
  if (ticket != last) return;
  // Online pass over the partials, four query heads of this KV head at a
  // time: lane l owns dims [l*DL, l*DL+DL) of each head.  The next partial's
  // loads are issued before the current one is folded in.
  constexpr int DL = D / 32;
  constexpr int GM = 4;
  const int G = p.group, H = kMQ ? p.num_queries * p.num_heads : p.num_heads;
  const int nq = kMQ ? p.num_queries : 1;
  for (int gq = 0, gn = 0; gq < G * nq; gq += gn) {
    // Rows of this KV head, at most four at a time and never across queries:
    // query qi, group heads g0 .. g0 + gn - 1.
    const int qi = gq / G, g0 = gq % G;
    const int h0 = qi * p.num_heads + kv_head * G + g0;
    gn = min(GM, G - g0);
    float run_m[GM], run_l[GM], acc[GM][DL];
    float nm[GM], nl[GM], no[GM][DL];
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      run_m[g] = -INFINITY;
      run_l[g] = 0.f;
#pragma unroll
      for (int i = 0; i < DL; ++i) acc[g][i] = 0.f;
    }
    auto load = [&](int rr) {
      const int sl = rr == r0 ? slot0 : 0;
      const size_t base = ((size_t)rr * 2 + sl) * H + h0;
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        if (g < gn) {
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + base + g);
          nm[g] = ml.x;
          nl[g] = ml.y;
          const float* po = p.part_o + (base + g) * D + lane * DL;
          if constexpr (DL == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(po));
            no[g][0] = v.x; no[g][1] = v.y; no[g][2] = v.z; no[g][3] = v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(po));
            no[g][0] = v.x; no[g][1] = v.y;
          }
        }
      }
    };
    load(r0);
    for (int rr = r0; rr <= r1; ++rr) {
      float cm[GM], cl[GM], co[GM][DL];
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        cm[g] = nm[g];
        cl[g] = nl[g];
#pragma unroll
        for (int i = 0; i < DL; ++i) co[g][i] = no[g][i];
      }
      if (rr < r1) load(rr + 1);
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        if (g < gn) {
          const float mnew = fmaxf(run_m[g], cm[g]);
          // Several queries: a query may have no keys in some (or all)
          // partials, m = -inf; keep -inf out of the exponent base.
          const float mb = (kMQ && mnew == -INFINITY) ? 0.f : mnew;
          const float a_old = ex2_ftz(run_m[g] - mb), a_new = ex2_ftz(cm[g] - mb);
          run_m[g] = mnew;
          run_l[g] = run_l[g] * a_old + cl[g] * a_new;
#pragma unroll
          for (int i = 0; i < DL; ++i) acc[g][i] = acc[g][i] * a_old + co[g][i] * a_new;
        }
      }
    }
    T* out = reinterpret_cast<T*>(p.out) + ((size_t)seq * H + h0) * D + lane * DL;
#pragma unroll
    for (int g = 0; g < GM; ++g) {
      if (g < gn) {
        const float inv = (kMQ && run_l[g] == 0.f) ? 0.f : p.v_scale / run_l[g];
#pragma unroll
        for (int i = 0; i < DL; ++i) out[(size_t)g * D + i] = T(acc[g][i] * inv);
      }
    }
  }
  __syncwarp();
  if (lane == 0) *cnt = 0;  // leave the counter zeroed for the next call
}

// A consumer warp that left its range before the end still takes the tickets of the cut
// sequences that it has not finished (`taken`: bit 0 the range's first one, in slot 0,
// bit 1 its last, in slot 1): with them every ticket gets all of its arrivals, and is back at
// zero when the call is over.  The call's output is unspecified then, as its error flag says.
// (By what the warp left in shared memory: with its place in a register until then 8 int8
// contexts of 32k took 107.4 us for 106.8.)
template <int WALK>
__device__ __forceinline__ void give_up_tickets(const DecodeParams& p, const long long* found, int r, int taken,
                                                int kv_head, int lane, int arrivals) {
  const int s = static_cast<int>(found[0]), S = p.num_seqs;
  const long long first = found[1], total = found[3], ranges = found[4];
  const long long a = range_start(r, total, ranges), b = range_start(r + 1, total, ranges);
  auto take = [&](long long lo, long long hi) {  // of a sequence of tiles lo .. hi - 1
    if (lane != 0 || segment_slot(a, b, lo, hi) < 0) return;
    const int r0 = static_cast<int>(range_of_tile(lo, total, ranges));
    const int r1 = static_cast<int>(range_of_tile(hi - 1, total, ranges));
    int* cnt = p.counters + (size_t)r0 * p.num_kv_heads + kv_head;
    if (atomicAdd(cnt, 1) == arrivals * (r1 - r0 + 1) - 1) *cnt = 0;
  };
  long long at = first + SeqWalk<WALK>(p, s, false).n;
  if ((taken & 1) == 0) take(first, at);
  if (at >= b || (taken & 2) != 0) return;
  for (int base = s + 1; base < S; base += 32) {
    const long long n = base + lane < S ? SeqWalk<WALK>(p, base + lane, false).n : 0;
    const long long hi = at + warp_incl_scan_ll(n, lane);
    const unsigned holds = __ballot_sync(0xffffffffu, hi - n < b && b <= hi);
    if (holds != 0) {
      const int from = __ffs(holds) - 1;
      const long long last = __shfl_sync(0xffffffffu, hi, from);
      take(last - __shfl_sync(0xffffffffu, n, from), last);
      return;
    }
    at = __shfl_sync(0xffffffffu, hi, 31);
  }
}
// As a call, for consumers at the register cap: 64 sequences x 4 queries of 32 heads on 8 take 111.2 us
// so, 113.4 with it written out; the others are faster without one (2 queries over int8 pools
// 70.2 for 71.6).
template <int WALK>
__device__ __noinline__ void give_up_tickets_call(const DecodeParams& p, const long long* found, int r, int taken,
                                                  int kv_head, int lane, int arrivals) {
  give_up_tickets<WALK>(p, found, r, taken, kv_head, lane, arrivals);
}

// One row of a cut sequence (kCutMerge), its partials added by log-sum-exp by a
// warp: lane i holds dims [i * D / 32, (i + 1) * D / 32).  The maxima and sums of up
// to 32 partials are read at once, one per lane, so that the loads of their O
// parts do not wait for one another.
template <int DL>
struct MergedRow {
  float m, l;
  float o[DL];
};

// With several warps per row, warp `part` of `parts` takes every parts-th partial.
template <int D>
__device__ __forceinline__ MergedRow<D / 32> merge_row(const float* part_ml, const float* part_o, const int4& cut,
                                                       int seq_rows, int in_seq, int lane, int part, int parts) {
  constexpr int DL = D / 32;
  MergedRow<DL> r;
  r.m = -INFINITY;
  r.l = 0.f;
#pragma unroll
  for (int i = 0; i < DL; ++i) r.o[i] = 0.f;
  // Range rr left its partial in slot 0, the first range in slot cut.z.
  auto at = [&](int rr) { return ((size_t)rr * 2 + (rr == cut.x ? cut.z : 0)) * seq_rows + in_seq; };
  for (int r0 = cut.x + part; r0 <= cut.y; r0 += 32 * parts) {
    const int rr = r0 + lane * parts;
    const float2 ml = rr <= cut.y ? __ldcg(reinterpret_cast<const float2*>(part_ml) + at(rr))
                                  : make_float2(-INFINITY, 0.f);
    float top = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float m = fmaxf(r.m, top), ref = m == -INFINITY ? 0.f : m;  // -inf: no token seen so far
    const float keep = ex2_ftz(r.m - ref), w = ex2_ftz(ml.x - ref);
    r.m = m;
    float l = w * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    r.l = r.l * keep + l;
#pragma unroll
    for (int i = 0; i < DL; ++i) r.o[i] *= keep;
    const int n = min(32, (cut.y - r0) / parts + 1);
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* po = part_o + at(r0 + k * parts) * D + lane * DL;
      if constexpr (DL == 4) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(po));
        r.o[0] = fmaf(wk, v.x, r.o[0]), r.o[1] = fmaf(wk, v.y, r.o[1]);
        r.o[2] = fmaf(wk, v.z, r.o[2]), r.o[3] = fmaf(wk, v.w, r.o[3]);
      } else {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(po));
        r.o[0] = fmaf(wk, v.x, r.o[0]), r.o[1] = fmaf(wk, v.y, r.o[1]);
      }
    }
  }
  return r;
}

// Appending calls: a tile holding some of the step's new tokens (tile rows
// mt.newfirst .. mt.nvalid - 1, query positions c - Q .. c - 1) may have been
// staged before those tokens reached the pool, so the warp of KV head kv_head
// puts each new token's K and V (from k_new / v_new, row s * Q + i for the
// token at position c - Q + i) into its own columns of the staged rows,
// swizzled as the tensor copy lays them out, and also stores them into the
// token's pool row (rows[r]; -1 leaves it unwritten).  Lane u < 16 moves
// 16-byte unit u of the K row, lane 16 + u the same unit of V.
template <int D>
__device__ __forceinline__ void append_new_rows(const DecodeParams& p, const StageMeta& mt, const int* rows,
                                                int kv_head, int w, uint32_t k_half, uint32_t v_half,
                                                int lane) {
  constexpr int UH = D * 2 / 16;  // 16-byte units of one head's bf16 row
  const int u = lane & 15;
  const bool is_v = lane >= 16;
  const int Q = p.num_queries;
  for (int r = mt.newfirst; r < mt.nvalid; ++r) {
    const int prow = rows[r];
    if (u < UH && prow >= 0) {
      const size_t tok = (size_t)mt.seq * Q + (mt.tok0 + r - (mt.ctx - Q));  // row of k_new / v_new
      const size_t e = (tok * p.num_kv_heads + kv_head) * D + u * 8;
      const uint4 val = __ldg(reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(is_v ? p.v_new : p.k_new) + e));
      const uint32_t unit = (uint32_t)(w * UH + u);
      const uint32_t L = (uint32_t)r * p.lines + (unit >> 3);
      const uint32_t dst = (is_v ? v_half : k_half) + L * kLine + (((unit & 7u) ^ (L & 7u)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(val.x), "r"(val.y),
                   "r"(val.z), "r"(val.w)
                   : "memory");
      __nv_bfloat16* pool = static_cast<__nv_bfloat16*>(const_cast<void*>(is_v ? p.v_cache : p.k_cache));
      *reinterpret_cast<uint4*>(pool + ((size_t)prow * p.num_kv_heads + kv_head) * D + u * 8) = val;
    }
  }
  // The stage is later refilled by the TMA engine (async proxy): order these
  // generic-proxy writes before that, and make them visible to the warp.
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// The same for FP8 pools (one query per sequence): the token's bf16 K/V are
// quantised exactly as the FP8 cache write does (fp32 quotient by the pool's
// scale, E4M3 round to nearest even, saturating), 16 codes per lane.
template <int D>
__device__ __forceinline__ void append_new_rows_fp8(const DecodeParams& p, const StageMeta& mt,
                                                    const int* rows, int kv_head, int w, uint32_t k_half,
                                                    uint32_t v_half, int lane) {
  constexpr int UH = D / 16;  // 16-byte units of one head's FP8 row
  const int u = lane & 15;
  const bool is_v = lane >= 16;
  const int Q = p.num_queries;
  for (int r = mt.newfirst; r < mt.nvalid; ++r) {
    const int prow = rows[r];
    if (u < UH && prow >= 0) {
      const size_t tok = (size_t)mt.seq * Q + (mt.tok0 + r - (mt.ctx - Q));
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(is_v ? p.v_new : p.k_new) + (tok * p.num_kv_heads + kv_head) * D +
          u * 16);
      const uint4 a = __ldg(src), b = __ldg(src + 1);
      const float sc = is_v ? p.v_scale : p.k_scale;
      const uint32_t in[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
            make_float2(bf16_lo(in[2 * i]) / sc, bf16_hi(in[2 * i]) / sc), __NV_SATFINITE, __NV_E4M3));
        const uint32_t hi = static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
            make_float2(bf16_lo(in[2 * i + 1]) / sc, bf16_hi(in[2 * i + 1]) / sc), __NV_SATFINITE, __NV_E4M3));
        out[i] = lo | (hi << 16);
      }
      const uint32_t unit = (uint32_t)(w * UH + u);
      const uint32_t L = (uint32_t)r * p.lines + (unit >> 3);
      const uint32_t dst = (is_v ? v_half : k_half) + L * kLine + (((unit & 7u) ^ (L & 7u)) << 4);
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst), "r"(out[0]), "r"(out[1]),
                   "r"(out[2]), "r"(out[3])
                   : "memory");
      unsigned char* pool = static_cast<unsigned char*>(const_cast<void*>(is_v ? p.v_cache : p.k_cache));
      *reinterpret_cast<uint4*>(pool + ((size_t)prow * p.num_kv_heads + kv_head) * D + u * 16) =
          make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

// ---------------------------------------------------------------------------
// Kernel 1
// ---------------------------------------------------------------------------
// QMODE 0: one query per sequence.  QMODE 1 / 2: several query tokens per
// sequence with a causal mask, (query, head) columns in one 8-wide MMA N-tile
// per warp: one warp per KV head (up to 8 columns) or p.split warps (2 to 4,
// up to 32 columns).
// WALK: which tiles, and what becomes of the rows (kWalkMod on the tensor-core
// paths: QMODE 1 or 2, also for one query).
// Walks other than kWalkAll keep to 128 registers where they can (four warps per
// quarter of an SM instead of three): their consumers wait on latency, and more of
// them hide it.  Rows of 128 dims need more: FP8 pools, 48 sequences x 4 queries take 74 us
// at 128 registers, with spills, and 56 at 168.
template <typename T, int D, int QMODE, int WALK>
constexpr int max_threads() {
  const bool fits = sizeof(T) == 2 && WALK != kWalkAll && (D == 64 || QMODE < 2);
  return fits ? 512 : 32 * (kMaxGroupHeads + kProducers);
}
template <typename T, int D, int GMAX, int QMODE, bool KV8 = false, int WALK = kWalkAll, bool I8 = false>
__global__ void __launch_bounds__(max_threads<T, D, QMODE, WALK>(), 1)
    pa_decode_kernel(const __grid_constant__ DecodeParams p) {
  extern __shared__ __align__(128) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nthreads = blockDim.x, nwarps = nthreads >> 5;
  const int HG = p.num_head_groups, R = p.num_ranges, S = p.num_seqs;
  const int r = blockIdx.x / HG, hg = blockIdx.x % HG;
  const int Hg = p.heads_per_cta;
  // QMODE 2 splits each KV head's (query, head) columns over p.split warps,
  // 8 columns each (up to 32 columns: four warps).
  const int kSplit = QMODE == 2 ? p.split : 1;
  constexpr bool kRows = QMODE == 2 && WALK != kWalkAll;  // 16 columns per warp, as rows
  const int NCW = Hg * kSplit;  // consumer warps; warps NCW .. NCW + producers - 1 produce
  const int producers = WALK == kWalkAll ? kProducers : nwarps - NCW;
  constexpr bool kMmaPath = (sizeof(T) == 2);  // tensor-core consumers, swizzled stages
  const Layout L = make_layout(p.stages, p.q_slots, p.q_bytes, p.stage_bytes, kMmaPath);
  long long* misc = reinterpret_cast<long long*>(smem + L.misc);  // [0,32) scratch, [32..] results
  if (WALK != kWalkRest || !p.beside)
    griddep_wait();  // inputs may come from the kernel just before (e.g. the cache write)

  // ---- Prologue: total tile count, this range, and its first sequence. ----
  long long total = 0;
  for (int base = 0; base < S; base += nthreads) {
    const int s = base + tid;
    long long n = (s < S) ? SeqWalk<WALK>(p, s, true).n : 0;
    if (s < S && n == 0 && s % gridDim.x == blockIdx.x) {
      if constexpr (WALK != kWalkAll) p.cuts[s] = make_int4(0, -1, 0, kCutEmpty);
      if constexpr (WALK != kWalkRest) zero_row<T, D>(p, s);
    }
    n = warp_sum_ll(n);
    if (lane == 0) misc[warp] = n;
    __syncthreads();
    for (int w = 0; w < nwarps; ++w) total += misc[w];
    __syncthreads();
  }
  // Never more ranges than tiles, so no range is empty and a cut sequence
  // has exactly r1 - r0 + 1 partials.
  long long Reff = total < R ? total : R;
  if constexpr (WALK == kWalkRest) {
    // The SMs the prefix kernel leaves.
    if (p.beside) {
      const int left = p.sm_count - prefix_share(p.prefix_units, total, S, HG,
                                                 walk_tile_us(p.row_bytes, p.group * p.num_queries),
                                                 p.num_queries * p.num_heads * D, D, p.sm_count);
      const long long most = static_cast<long long>(left) * R / p.sm_count;
      Reff = min(Reff, max(most, 1ll));
    }
  }
  if (r >= Reff) {
    if (WALK == kWalkRest && p.beside) griddep_wait();
    return;
  }
  const long long a = range_start(r, total, Reff), b = range_start(r + 1, total, Reff);

  long long run = 0;
  for (int base = 0; base < S; base += nthreads) {
    const int s = base + tid;
    const long long n = (s < S) ? SeqWalk<WALK>(p, s, false).n : 0;
    const long long incl = warp_incl_scan_ll(n, lane);
    if (lane == 31) misc[warp] = incl;
    __syncthreads();
    long long before = run;
    for (int w = 0; w < warp; ++w) before += misc[w];
    long long chunk = 0;
    for (int w = 0; w < nwarps; ++w) chunk += misc[w];
    const long long excl = before + incl - n;
    if (s < S && n > 0 && excl <= a && a < excl + n) {
      misc[32] = s;
      misc[33] = excl;
    }
    if constexpr (WALK != kWalkAll) {
      if (s < S && n > 0 && s % (Reff * HG) == blockIdx.x) {
        const int r0 = static_cast<int>(range_of_tile(excl, total, Reff));
        const int r1 = static_cast<int>(range_of_tile(excl + n - 1, total, Reff));
        p.cuts[s] = make_int4(r0, r1, partial_slot_of_range(r0, excl, total, Reff), r0 == r1 ? kCutWhole : kCutMerge);
      }
    }
    run += chunk;
    __syncthreads();
  }
  griddep_launch_dependents();  // the next kernel may get resident; it waits for our completion

  const uint32_t bar0 = smem_addr(smem + L.bar);
  const int NS = p.stages, NQ = p.q_slots;
  auto full_bar = [&](int i) { return bar0 + 8u * i; };
  auto empty_bar = [&](int i) { return bar0 + 8u * (NS + i); };
  auto qfull_bar = [&](int i) { return bar0 + 8u * (2 * NS + i); };
  auto qempty_bar = [&](int i) { return bar0 + 8u * (2 * NS + NQ + i); };
  StageMeta* meta = reinterpret_cast<StageMeta*>(smem + L.meta);
  int* stage_rows = reinterpret_cast<int*>(smem + L.rows);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 34);
  // A pipeline wait ran out: report it and tell the producers to drain.
  auto timed_out = [&]() {
    if (lane == 0) {
      report(p.error_flag, PA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  // A stage or a walk is not where it should be: say so and leave instead of
  // taking a sequence or range from it as an index into global memory.
  auto lost = [&]() {
    if (lane == 0) {
      report(p.error_flag, PA_DEVERR_STATE);
      *abort_flag = 1;
    }
  };
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full_bar(i), I8 ? 33 : 1);  // int8: and the lanes' copies of scales
      mbar_init(empty_bar(i), NCW);
    }
    for (int i = 0; i < NQ; ++i) {
      mbar_init(qfull_bar(i), 1);
      mbar_init(qempty_bar(i), NCW);
    }
    *abort_flag = 0;
    misc[35] = total;  // (give_up_tickets)
    misc[36] = Reff;
    misc[37] = misc[38] = 0;
    mbar_init_fence();
  }
  __syncthreads();
  const int s_first = static_cast<int>(misc[32]);
  const long long p_first = misc[33];
  const uint32_t q_slot_bytes = (p.q_bytes + 127u) & ~127u;
  const uint32_t qring = smem_addr(smem + L.qring);
  const uint32_t stages =
      kMmaPath ? ((smem_addr(smem + L.stage) + 1023u) & ~1023u) : smem_addr(smem + L.stage);
  const int G = p.group, H = p.num_heads, Hk = p.num_kv_heads, bs = p.block_size;

  if (warp >= NCW) {
    // ---------------- producers ----------------
    const int pw = warp - NCW;  // this producer takes the tiles x with (x - a) % kProducers == pw
    // Pool element: T, or one byte for an FP8 pool.
    using KV = typename std::conditional<KV8, unsigned char, T>::type;
    const KV* kc = reinterpret_cast<const KV*>(p.k_cache);
    const KV* vc = reinterpret_cast<const KV*>(p.v_cache);
    const T* qg = reinterpret_cast<const T*>(p.q);
    int s = s_first;
    long long ps = p_first;
    SeqWalk<WALK> sw(p, s, false);
    int c = sw.c;
    long long ns = sw.n;
    // The next sequence's length is fetched one sequence ahead.
    SeqWalk<WALK> sw_next;
    if (s + 1 < S) sw_next = SeqWalk<WALK>(p, s + 1, false);
    int slot = 0, seg_r0 = 0, seg_r1 = 0, seg_slot0 = 0;
    int st = 0, qi = 0;
    uint32_t ph = 0, qph = 0;
    // Stages and query slots this warp armed, with the parity of the last
    // phase it armed on each (for the drain after a timeout).
    uint32_t my_stages = 0u, my_stage_par = 0u, my_qs = 0u, my_q_par = 0u;
    const int t = lane & 15;
    const bool is_v = lane >= 16;
    if (kMmaPath && lane == 0) {
      prefetch_tensormap(&p.tm_k);
      prefetch_tensormap(&p.tm_v);
    }
    // Per-lane constants of the copy issue: whether this lane leads a copy
    // (tensor paths: the first row of a box), where in a stage its copy
    // lands, and which pool it reads.  Power-of-two block sizes take shifts
    // and masks instead of integer division.
    const bool lead = kMmaPath ? (t % (int)p.box_rows) == 0 : true;
    const uint32_t lane_dst = kMmaPath ? (is_v ? kTile * p.lines * kLine : 0u) + t * p.lines * kLine
                                       : (is_v ? kTile * p.pitch : 0u) + t * p.pitch;
    const void* tmap = is_v ? static_cast<const void*>(&p.tm_v) : static_cast<const void*>(&p.tm_k);
    const int bs_sh = (bs & (bs - 1)) == 0 ? __ffs(bs) - 1 : -1;
    auto blk_of = [&](int tok) { return bs_sh >= 0 ? tok >> bs_sh : tok / bs; };
    auto off_of = [&](int tok) { return bs_sh >= 0 ? tok & (bs - 1) : tok % bs; };
    // Block-table window of the current sequence: lane i holds entry cb+i in
    // `cur` and cb+32+i in `nxt`.  The window slides one chunk at a time and the
    // next chunk is loaded a chunk ahead, so lookups never wait on memory except
    // at the first tile of a segment.
    const int32_t* bt_row = nullptr;
    int nblk = 0, cb = 0, cur = -1, nxt = -1;
    bool bad_ids = false;  // block ids outside the pool among this lane's
    auto table_entry = [&](int idx) -> int { return idx < nblk ? __ldg(bt_row + idx) : -1; };
    for (long long x = a; x < b; ++x) {
      bool new_seq = (x == a);
      while (x >= ps + ns && s < S) {
        ps += ns;
        ++s;
        sw = sw_next;
        c = sw.c;
        ns = sw.n;
        sw_next = SeqWalk<WALK>();
        if (s + 1 < S) sw_next = SeqWalk<WALK>(p, s + 1, false);
        new_seq = true;
      }
      if (s >= S) {
        lost();
        break;
      }
      const int j = static_cast<int>(x - ps);
      const int tok0 = sw.token(j);
      int nvalid = min(kTile, c - tok0);
      if constexpr (WALK == kWalkMod) nvalid = __ballot_sync(0xffffffffu, sw.sees(tok0 + t)) & 0xffff;
      const int blk0 = blk_of(tok0);
      if (new_seq) {
        slot = segment_slot(a, b, ps, ps + ns);
        if (slot >= 0) {
          seg_r0 = static_cast<int>(range_of_tile(ps, total, Reff));
          seg_r1 = static_cast<int>(range_of_tile(ps + ns - 1, total, Reff));
          seg_slot0 = partial_slot_of_range(seg_r0, ps, total, Reff);
        }
        bt_row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
        nblk = (c + bs - 1) / bs;
        cb = blk0;
        cur = table_entry(cb + lane);
        nxt = table_entry(cb + 32 + lane);
      }
      while (blk0 >= cb + 32) {
        if (WALK == kWalkMod && blk0 >= cb + 96) {  // from the prefix to the window: start afresh
          cb = blk0;
          cur = table_entry(cb + lane);
          nxt = table_entry(cb + 32 + lane);
          break;
        }
        cur = nxt;
        cb += 32;
        nxt = table_entry(cb + 32 + lane);
      }
      const int flags = (new_seq ? kSegBegin : 0) | ((x == b - 1 || j == ns - 1) ? kSegEnd : 0) |
                        ((slot + 1) << 2) | (seg_slot0 << 4) | tile_tag(x);
      const bool mine = static_cast<int>((x - a) % (WALK == kWalkAll ? kProducers : producers)) == pw;
      // One producer fills all query slots, whoever takes the sequence's first tile:
      // it sees every phase of a slot's barrier, so that the parity it waits for is
      // never an older or a later phase's.  (Had the owner of the first tile filled it, a
      // producer that skipped sequences of few tiles could be two phases ahead at its
      // next own one; one that waited without filling could come a phase too late.)
      if (new_seq && pw == 0) {
        if (!mbar_wait_warp(qempty_bar(qi), qph ^ 1u, p.wait_limit_ns)) {
          timed_out();
          break;
        }
        if (lane == 0) {
          const uint32_t qb = qfull_bar(qi);
          mbar_arrive_expect_tx(qb, p.q_bytes);
          if constexpr (QMODE == 0) {
            bulk_copy_g2s(qring + qi * q_slot_bytes, qg + ((size_t)s * H + (size_t)hg * Hg * G) * D,
                          p.q_bytes, qb);
          } else {
            // Query rows are [seq][query][head]: one copy per query token.
            const uint32_t per_q = p.q_bytes / p.num_queries;
            for (int qq = 0; qq < p.num_queries; ++qq)
              bulk_copy_g2s(qring + qi * q_slot_bytes + qq * per_q,
                            qg + (((size_t)s * p.num_queries + qq) * H + (size_t)hg * Hg * G) * D,
                            per_q, qb);
          }
        }
        my_qs |= 1u << qi;
        my_q_par = (my_q_par & ~(1u << qi)) | (qph << qi);
      }
      if (new_seq && ++qi == NQ) {  // every producer follows the query ring
        qi = 0;
        qph ^= 1u;
      }
      if (!mine) {  // the other producer's tile: only follow the stage ring
        if (++st == NS) {
          st = 0;
          ph ^= 1u;
        }
        continue;
      }
      // This lane's token -> physical block (a tile spans at most 16 blocks, so
      // it always lies inside the 64-entry window).
      const int tok = tok0 + t;
      const int rel = blk_of(tok) - cb;
      const int e_cur = __shfl_sync(0xffffffffu, cur, rel & 31);
      const int e_nxt = __shfl_sync(0xffffffffu, nxt, rel & 31);
      const int phys = rel < 32 ? e_cur : e_nxt;
      bool ok = t < nvalid;
      // A box is copied if some query sees one of its rows.
      if constexpr (WALK == kWalkMod)
        ok = lead && ((nvalid >> t) & (kMmaPath ? (1 << p.box_rows) - 1 : 1)) != 0;
      // Reported behind the loop: a branch here would be on the way of every tile's copies.
      const bool bad =
          ok && p.num_physical_blocks > 0 && static_cast<unsigned>(phys) >= static_cast<unsigned>(p.num_physical_blocks);
      bad_ids |= bad;
      ok = ok && !bad;
      // Tensor-core paths: lane t (t a multiple of box_rows) copies tile rows
      // t .. t + box_rows - 1, which lie in one block, as one tensor box; rows
      // past the context in that block come along and are masked by the
      // consumers.  fp32: one bulk copy per valid token row.
      ok = ok && lead;
      const unsigned copies = __ballot_sync(0xffffffffu, ok);
      // Token row of the pool: fewer than 2^31 in any pool that fits in device memory.
      const int row = (int)((bs_sh >= 0 ? (unsigned)phys << bs_sh : (unsigned)phys * (unsigned)bs) +
                            (unsigned)off_of(tok));
      // Appending calls: the step's new tokens are positions c - Q .. c - 1.
      int newfirst = -1;
      if (WALK == kWalkAll && kMmaPath && p.k_new != nullptr && tok0 + nvalid > c - p.num_queries) {
        newfirst = max(0, c - p.num_queries - tok0);
      }
      if (!mbar_wait_warp(empty_bar(st), ph ^ 1u, p.wait_limit_ns)) {
        timed_out();
        break;
      }
      // Tests of the bounded waits: this tile's stage is never armed or
      // filled, so the consumers' wait on it runs out.
      const bool stall = x == p.stall_tile;
      if (WALK == kWalkAll && newfirst >= 0 && !is_v && t >= newfirst && t < nvalid) {
        // Pool row of this tile row's new token; a failed block check leaves it unwritten.
        const bool none = p.num_physical_blocks > 0 && (phys < 0 || phys >= p.num_physical_blocks);
        stage_rows[st * kTile + t] = none ? -1 : row;
      }
      __syncwarp();
      if (lane == 0 && !stall) {
        meta[st] = StageMeta{s, tok0, nvalid, flags, seg_r0, seg_r1, c, WALK == kWalkMod ? sw.pre : newfirst};
        mbar_arrive_expect_tx(full_bar(st), __popc(copies) * (kMmaPath ? p.box_bytes : p.row_bytes));
      }
      __syncwarp();
      if (!stall) {
        my_stages |= 1u << st;
        my_stage_par = (my_stage_par & ~(1u << st)) | (ph << st);
      }
      if (ok && !stall) {
        const uint32_t dst = stages + st * p.stage_bytes + lane_dst;
        if constexpr (WALK == kWalkRest) {  // read once: leave L2 to the prefix
          tma_load_4d_hint(dst, tmap, 0, 0, hg, row, full_bar(st), l2_evict_first());
        } else if constexpr (kMmaPath) {
          tma_load_4d(dst, tmap, 0, 0, hg, row, full_bar(st));
        } else {
          const KV* src = (is_v ? vc : kc) + ((size_t)row * Hk + (size_t)hg * Hg) * D;
          bulk_copy_g2s(dst, src, p.row_bytes, full_bar(st));
        }
      }
      if constexpr (I8) {
        // The scales of the tile's rows, 4 rows of a block at a time where its size allows.
        if (!stall) {
          const uint32_t to = stages + st * p.stage_bytes + 2 * kTile * p.lines * kLine;
          auto copy_scales = [&](auto rows_tag) {
            constexpr int kRows = decltype(rows_tag)::value;
            const int runs = kTile / kRows * Hg;  // of K; then V's
            for (int i0 = 0; i0 < 2 * runs; i0 += 32) {
              const int i = i0 + lane, v = i >= runs, j = v ? i - runs : i;
              const int head = j / (kTile / kRows), t0 = j % (kTile / kRows) * kRows;
              const int blk = __shfl_sync(0xffffffffu, phys, t0);
              if (i < 2 * runs) {
                const bool there = t0 < nvalid && !(p.num_physical_blocks > 0 && static_cast<unsigned>(blk) >=
                                                                                    static_cast<unsigned>(p.num_physical_blocks));
                const float* src = (v ? p.v_scales : p.k_scales) +
                                   ((size_t)(there ? blk : 0) * Hk + hg * Hg + head) * bs + off_of(tok0 + t0);
                const uint32_t dst = to + 4u * ((v * Hg + head) * kTile + t0);
                if constexpr (kRows == 4)
                  copy_async16(dst, src, there);
                else
                  copy_async4(dst, src, there);
              }
            }
          };
          if ((bs & 3) == 0)
            copy_scales(std::integral_constant<int, 4>{});
          else
            copy_scales(std::integral_constant<int, 1>{});
          copies_arrive(full_bar(st));
        }
      }
      if (++st == NS) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (bad_ids) report(p.error_flag, PA_DEVERR_BLOCK_ID);
    named_barrier_sync(1, nthreads);  // every warp has left its tile loop
    if (*abort_flag != 0 && lane == 0) {
      // A wait ran out, so the loops ended early and copies this warp started
      // may still be landing.  Wait (again bounded) for the last phase it
      // armed on each stage and query slot, so that no copy writes into this
      // CTA's shared memory after it has retired.
      for (int i = 0; i < NS; ++i)
        if ((my_stages >> i) & 1u) (void)mbar_wait(full_bar(i), (my_stage_par >> i) & 1u, p.wait_limit_ns);
      for (int i = 0; i < NQ; ++i)
        if ((my_qs >> i) & 1u) (void)mbar_wait(qfull_bar(i), (my_q_par >> i) & 1u, p.wait_limit_ns);
    }
  } else {
    // ---------------- consumers ----------------
    const int w = warp / kSplit;  // KV head within the group
    const int col_base = (warp % kSplit) * (kRows ? 16 : 8);
    const int kv_head = hg * Hg + w;
    int st = 0, qi = 0;
    uint32_t ph = 0, qph = 0;
    constexpr bool kMma = (sizeof(T) == 2);
    constexpr bool kMod = WALK == kWalkMod;
    using Mma = typename std::conditional<
        KV8, MmaConsumerF8<D, (QMODE > 0), kMod, I8>,
        typename std::conditional<QMODE == 0, MmaConsumer<D>, MmaConsumerMQ<D, 1, kMod>>::type>::type;
    using Columns = typename std::conditional<kRows, RowsConsumer<D, KV8, kMod>, Mma>::type;
    using Simt = typename std::conditional<kMod, Fp32ModConsumer<D, GMAX>, SimtConsumer<D, GMAX>>::type;
    constexpr bool kFp32Mod = kMod && !kMma;
    typename std::conditional<kMma, Columns, Simt>::type cons;
    float2* weights = nullptr;
    if constexpr (kFp32Mod) {
      __shared__ float2 weight_buffers[kMaxGroupHeads][(kTile + 1) * GMAX];
      static_assert(sizeof(weight_buffers) <= kFp32Buffers, "the host plan leaves room for them");
      weights = weight_buffers[warp];
      cons.setup(p, kv_head, lane);
    }
    if constexpr (kRows) {
      cons.setup(p, kv_head, col_base, w, lane);
    } else {
      if constexpr (KV8) cons.setup(p.lines, w * D / 16, lane);
      if constexpr (kMod && kMma) cons.mc.setup(p, kv_head, col_base + 2 * (lane & 3));
    }
    // FP8 consumers, and bf16 ones that split a KV head's columns over
    // several warps, take two stages at a time when both hold the same
    // segment (tile pairing: tile2), if the ring has four or more stages.
    // Their tile math, not HBM, sets the pace.  One-query bf16 decode and
    // bf16 multi-query with one warp per KV head (2 KiB rows, a 3-stage ring
    // for the common shapes) are HBM-bound and keep the ring for copies.
    constexpr bool kPair = kMma && (KV8 || QMODE == 2);
    // Whether a stage holds tile x, of a sequence of the batch: asked where the stage's
    // sequence becomes an address, not for every tile (which cost 96 sequences x 3 queries of
    // 6 x 64 dims, at their 128 registers, 80 us instead of 72).
    auto in_place = [S](const StageMeta& m, long long x) {
      return tag_matches(m.flags, x) && static_cast<unsigned>(m.seq) < static_cast<unsigned>(S);
    };
    // Rows of a tile to attend: the walk's mask, or the first nvalid.
    auto tile_mask = [](int nvalid) -> uint32_t {
      return kMod ? (uint32_t)nvalid : nvalid < kTile ? (1u << nvalid) - 1u : 0xffffu;
    };
    for (long long x = a; x < b; ++x) {
      if (!mbar_wait_warp(full_bar(st), ph, p.wait_limit_ns)) {
        timed_out();
        break;
      }
      const StageMeta mt = meta[st];
      if (mt.flags & kSegBegin) {
        if (!mbar_wait_warp(qfull_bar(qi), qph, p.wait_limit_ns)) {
          timed_out();
          break;
        }
        if constexpr (kFp32Mod)
          cons.begin_segment(smem + L.qring + qi * q_slot_bytes, w, G);
        else if constexpr (kRows)
          cons.begin_segment(p, smem + L.qring + qi * q_slot_bytes, w, lane);
        else if constexpr (QMODE == 0)
          cons.begin_segment(smem + L.qring + qi * q_slot_bytes, w, G, lane);
        else if constexpr (KV8)
          cons.begin_segment(smem + L.qring + qi * q_slot_bytes, w, G, lane, p.num_queries, Hg, col_base);
        else
          cons.begin_segment(smem + L.qring + qi * q_slot_bytes, w, G, p.num_queries, Hg, lane,
                             col_base);
        if constexpr (!kFp32Mod) {  // that one reads the queries in place, until the segment ends
          __syncwarp();
          if (lane == 0) mbar_arrive(qempty_bar(qi));
          if (++qi == NQ) {
            qi = 0;
            qph ^= 1u;
          }
        }
      }
      constexpr int kKVBytes = KV8 ? 1 : (int)sizeof(T);
      const uint32_t k_half = stages + st * p.stage_bytes;
      const uint32_t v_half = k_half + kTile * p.lines * kLine;
      const int uh = w * D * kKVBytes / 16;  // this head's first 16-byte unit in the row
      auto scales_of = [&](int stage) {  // int8
        return reinterpret_cast<const float*>(smem + (stages - smem_addr(smem)) + stage * p.stage_bytes +
                                              2 * kTile * p.lines * kLine) + w * kTile;
      };
      if constexpr (I8) {
        cons.scales = scales_of(st);
        cons.v_scales_at = Hg * kTile;
      }
      if constexpr (kMma && QMODE < 2 && WALK == kWalkAll && !I8) {
        if (mt.newfirst >= 0) {
          if (!in_place(mt, x)) {
            lost();
            break;
          }
          const int* rows = stage_rows + st * kTile;
          if constexpr (KV8)
            append_new_rows_fp8<D>(p, mt, rows, kv_head, w, k_half, v_half, lane);
          else
            append_new_rows<D>(p, mt, rows, kv_head, w, k_half, v_half, lane);
        }
      }
      // A tile that does not end its segment is followed, in the next stage,
      // by the same segment's next tile: pair them.
      bool paired = false;
      StageMeta me = mt;  // the pass's last tile (it carries the segment end)
      int st_last = st;
      if constexpr (kPair) {
        // The ring has four or more stages here (the host plan checks it): a
        // pair holds two, and the copies need the rest.
        if (!(mt.flags & kSegEnd)) {
          const int st2 = st + 1 == NS ? 0 : st + 1;
          const uint32_t ph2 = st + 1 == NS ? ph ^ 1u : ph;
          if (!mbar_wait_warp(full_bar(st2), ph2, p.wait_limit_ns)) {
            timed_out();
            break;
          }
          me = meta[st2];
          const uint32_t k_half2 = stages + st2 * p.stage_bytes;
          const uint32_t v_half2 = k_half2 + kTile * p.lines * kLine;
          if constexpr (QMODE < 2 && WALK == kWalkAll && !I8) {
            if (me.newfirst >= 0) {
              if (!in_place(me, x + 1)) {
                lost();
                break;
              }
              if constexpr (KV8)
                append_new_rows_fp8<D>(p, me, stage_rows + st2 * kTile, kv_head, w, k_half2, v_half2, lane);
              else
                append_new_rows<D>(p, me, stage_rows + st2 * kTile, kv_head, w, k_half2, v_half2, lane);
            }
          }
          const ModTile mo0{tile_mask(mt.nvalid), mt.tok0, mt.ctx, mt.newfirst};
          const ModTile mo1{tile_mask(me.nvalid), me.tok0, me.ctx, me.newfirst};
          if constexpr (kRows)
            cons.template tiles<2>(p, {k_half, k_half2}, {v_half, v_half2}, uh, {mo0, mo1}, lane);
          else if constexpr (kMod && KV8)
            cons.tile2(k_half, v_half, k_half2, v_half2, 0, p.scale_log2, lane, mt.tok0, mt.ctx, G,
                       p.num_queries, &p, mo0, mo1);
          else if constexpr (I8)
            cons.tile2(k_half, v_half, k_half2, v_half2, me.nvalid, p.scale_log2, lane, mt.tok0, mt.ctx, G,
                       p.num_queries, nullptr, ModTile(), ModTile(), scales_of(st2));
          else if constexpr (KV8 && QMODE > 0)
            cons.tile2(k_half, v_half, k_half2, v_half2, me.nvalid, p.scale_log2, lane, mt.tok0, mt.ctx, G,
                       p.num_queries);
          else if constexpr (KV8)
            cons.tile2(k_half, v_half, k_half2, v_half2, me.nvalid, p.scale_log2, lane);
          else
            cons.tile2(k_half, v_half, k_half2, v_half2, p.lines, uh, me.nvalid, mt.tok0, mt.ctx, G,
                       p.num_queries, p.scale_log2, lane);
          paired = true;
          st_last = st2;
          ++x;
        }
      }
      const ModTile mo{tile_mask(mt.nvalid), mt.tok0, mt.ctx, mt.newfirst};
      if (paired) {
      } else if constexpr (kRows) {
        cons.template tiles<1>(p, {k_half}, {v_half}, uh, {mo}, lane);
      } else if constexpr (kMod && KV8) {
        cons.tile(k_half, v_half, 0, p.scale_log2, lane, mt.tok0, mt.ctx, G, p.num_queries, &p, mo);
      } else if constexpr (kMod && kMma) {
        cons.tile(k_half, v_half, p.lines, uh, 0, mt.tok0, mt.ctx, G, p.num_queries, p.scale_log2, lane, &p, mo);
      } else if constexpr (kMod) {
        const unsigned char* kb = smem + L.stage + st * p.stage_bytes + w * D * sizeof(T);
        cons.tile(p, kb, kb + kTile * p.pitch, mo, weights, lane);
      } else if constexpr (KV8 && QMODE > 0) {
        cons.tile(k_half, v_half, mt.nvalid, p.scale_log2, lane, mt.tok0, mt.ctx, G, p.num_queries);
      } else if constexpr (KV8) {
        cons.tile(k_half, v_half, mt.nvalid, p.scale_log2, lane);
      } else if constexpr (kMma && QMODE == 2) {
        cons.tile_hoisted(k_half, v_half, p.lines, uh, mt.nvalid, mt.tok0, mt.ctx, G, p.num_queries,
                          p.scale_log2, lane);
      } else if constexpr (kMma && QMODE > 0) {
        cons.tile(k_half, v_half, p.lines, uh, mt.nvalid, mt.tok0, mt.ctx, G, p.num_queries,
                  p.scale_log2, lane);
      } else if constexpr (kMma) {
        cons.tile(k_half, v_half, p.lines, uh, mt.nvalid, p.scale_log2, lane);
      } else {
        const unsigned char* kb = smem + L.stage + st * p.stage_bytes + w * D * sizeof(T);
        cons.tile(kb, kb + kTile * p.pitch, p.pitch, mt.nvalid, p.scale_log2, G, lane);
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(empty_bar(st));
        if (paired) mbar_arrive(empty_bar(st_last));
      }
      if (me.flags & kSegEnd) {
        if constexpr (kFp32Mod) {
          if (lane == 0) mbar_arrive(qempty_bar(qi));
          if (++qi == NQ) {
            qi = 0;
            qph ^= 1u;
          }
        }
        const int slot = ((me.flags >> 2) & 3) - 1;
        if (!in_place(me, x) || slot > 1 || (WALK == kWalkAll && slot >= 0 && (me.r0 < 0 || me.r0 > r || me.r1 < r || me.r1 >= R || me.r0 == me.r1))) {
          lost();
          break;
        }
        if constexpr (WALK == kWalkRest)
          cons.template finish<true>(p, me.seq, kv_head, slot, r, lane);
        else
          cons.finish(p, me.seq, kv_head, slot, r, lane);
        if (WALK == kWalkAll && slot >= 0) {
          if (lane == 0) reinterpret_cast<unsigned char*>(misc + 37)[warp] |= 1u << slot;
          arrive_and_merge<T, D, (QMODE > 0)>(p, me.seq, kv_head, me.r0, me.r1, (me.flags >> 4) & 1, lane,
                                              kSplit);
        }
        // Split-column kernels sit at the register cap: writing the state here
        // (the next segment's begin_segment rewrites it anyway) frees its
        // registers for the merge above.
        if constexpr (QMODE == 2 && !kRows) cons.clear();
      }
      if (++st == NS) {
        st = 0;
        ph ^= 1u;
      }
      if (paired && ++st == NS) {
        st = 0;
        ph ^= 1u;
      }
    }
    named_barrier_sync(1, nthreads);  // lets the producers drain their copies after a timeout
    if (WALK == kWalkAll && *abort_flag != 0) {
      const int taken = reinterpret_cast<unsigned char*>(misc + 37)[warp];
      if constexpr (QMODE == 2)
        give_up_tickets_call<WALK>(p, misc + 32, r, taken, kv_head, lane, kSplit);
      else
        give_up_tickets<WALK>(p, misc + 32, r, taken, kv_head, lane, kSplit);
    }
  }
  if (WALK == kWalkRest && p.beside) griddep_wait();
  (void)Hk;
}

}  // namespace pa
