// Work decomposition of one decode batch, shared by the attention kernel, the
// merge kernel and host-side tests (plain C++ when compiled without nvcc).
//
// Every sequence s contributes ceil(ctx_s / kTile) tiles of kTile tokens.  The
// tiles of all sequences, in sequence order, form one flat list of T tiles.
// That list is cut into R equal ranges: range r owns tiles
// [floor(r*T/R), floor((r+1)*T/R)).  One CTA (per KV-head group) walks one
// range, so every CTA streams the same number of K/V bytes whatever the
// context-length mix.  A sequence whose tiles all fall in one range is
// finished by that CTA; a sequence that straddles ranges leaves one partial
// result per range it touches, merged afterwards by log-sum-exp.
//
// Partial-result slot rule: in range r, the sequence holding the range's first
// tile writes slot 0; a different sequence cut at the range's end writes slot
// 1.  Every other sequence touched by the range lies wholly inside it.
#pragma once

#include <stdint.h>

#if defined(__CUDACC__)
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

constexpr int kTile = 16;  // tokens per tile (one MMA M-extent, one pipeline stage)

PA_HD int64_t range_start(int64_t r, int64_t total_tiles, int64_t num_ranges) {
  const int64_t prod = r * total_tiles;
  // 32-bit division when the operands fit (the common case; much cheaper on the GPU).
  if (prod < (int64_t(1) << 32) && num_ranges < (int64_t(1) << 32))
    return static_cast<int64_t>(static_cast<uint32_t>(prod) / static_cast<uint32_t>(num_ranges));
  return prod / num_ranges;
}

// The range that owns tile x (0 <= x < total_tiles).  Empty ranges own nothing.
PA_HD int64_t range_of_tile(int64_t x, int64_t total_tiles, int64_t num_ranges) {
  const int64_t prod = x * num_ranges;
  int64_t r = (prod < (int64_t(1) << 32) && total_tiles < (int64_t(1) << 32))
                  ? static_cast<int64_t>(static_cast<uint32_t>(prod) / static_cast<uint32_t>(total_tiles))
                  : prod / total_tiles;
  if (r >= num_ranges) r = num_ranges - 1;
  while (r + 1 < num_ranges && range_start(r + 1, total_tiles, num_ranges) <= x) ++r;
  while (r > 0 && range_start(r, total_tiles, num_ranges) > x) --r;
  return r;
}

PA_HD int tiles_of(int ctx) { return (ctx + kTile - 1) / kTile; }

// Output destination of the segment [seg_lo, seg_hi) of a sequence whose tiles
// are [seq_lo, seq_hi), walked by the range [r_lo, r_hi).
//   -1: the whole sequence is in this range (write the final output);
//    0 / 1: partial slot.
PA_HD int segment_slot(int64_t r_lo, int64_t r_hi, int64_t seq_lo, int64_t seq_hi) {
  if (r_lo <= seq_lo && r_hi >= seq_hi) return -1;
  return (r_lo >= seq_lo) ? 0 : 1;
}

// Slot in which range r left its partial for a sequence starting at tile
// seq_lo (r must touch that sequence and be non-empty).
PA_HD int partial_slot_of_range(int64_t r, int64_t seq_lo, int64_t total_tiles,
                                int64_t num_ranges) {
  return (range_start(r, total_tiles, num_ranges) >= seq_lo) ? 0 : 1;
}

// Whole token rows from address `at` to the end of the allocation [start, start + size)
// (0 if it does not hold the address), at most 2^31.
PA_HD uint64_t rows_behind(uint64_t start, uint64_t size, uint64_t at, uint64_t row_bytes) {
  if (at < start || at - start >= size) return 0;
  const uint64_t rows = (size - (at - start)) / row_bytes;
  return rows < (uint64_t(1) << 31) ? rows : uint64_t(1) << 31;
}

// Which tiles of a sequence a kernel walks, and what becomes of its rows.
enum : int {
  kWalkAll = 0,   // every token, plain scores, output rows
  kWalkMod = 1,   // the tiles some query sees, modified scores, output rows
  kWalkRest = 2,  // the tokens behind a shared prefix, plain scores, (m, l, O) rows
};
constexpr int kNoWindow = 1 << 30;  // longer than any context

// The tiles a sequence of c tokens contributes.  kWalkMod: `nh` tiles from token
// h0 (the prefix every query sees), then the tiles from token t0 (what the window
// leaves, from the first query's); kWalkRest: tiles from token t0.  A token is
// seen by some query if it is in [first, pre) or in [max(first, lo), c).
template <int WALK>
struct SeqSpan {
  int c = 0, n = 0;
  int nh = 0, h0 = 0, t0 = 0, first = 0, pre = 0, lo = 0;

#if defined(__CUDA_ARCH__)
  PA_HD static int smaller(int a, int b) { return min(a, b); }
  PA_HD static int larger(int a, int b) { return max(a, b); }
#else
  PA_HD static int smaller(int a, int b) { return a < b ? a : b; }
  PA_HD static int larger(int a, int b) { return a > b ? a : b; }
#endif

  PA_HD void all(int context) {
    c = context;
    n = tiles_of(c);
  }
  PA_HD void rest(int context, int prefix_tokens, int num_queries) {
    c = context;
    t0 = c >= prefix_tokens + num_queries - 1 ? prefix_tokens : 0;
    n = tiles_of(c - t0);
  }
  PA_HD void seen(int context, int first_token, int prefix_len, int num_queries, int window) {
    c = context;
    first = larger(0, first_token);
    pre = larger(0, smaller(c, prefix_len));
    // The first query that exists sees back to its position - window + 1.
    lo = larger(larger(first, pre), larger(0, c - num_queries) - window + 1);
    if (first < c) {
      h0 = first & ~(kTile - 1);
      nh = pre > first ? tiles_of(pre - h0) : 0;
      t0 = larger(lo & ~(kTile - 1), nh > 0 ? h0 + nh * kTile : 0);
      n = nh + (c > t0 ? tiles_of(c - t0) : 0);
    }
  }
  PA_HD int token(int j) const {
    if (WALK == kWalkAll) return j * kTile;
    if (WALK == kWalkRest) return t0 + j * kTile;
    return j < nh ? h0 + j * kTile : t0 + (j - nh) * kTile;
  }
  PA_HD bool sees(int tok) const {  // kWalkMod
    return tok < c && tok >= first && (tok < pre || tok >= lo);
  }
};

// SeqCut, what the walks other than kWalkAll leave per sequence: (first range,
// last range, slot of the first range's partial, state).
enum : int { kCutEmpty = 0, kCutWhole = 1, kCutMerge = 2 };

// Whether the cut of a sequence names partials of `ranges` ranges.  The kernels that
// add the partials ask before they use one as an index.
PA_HD bool cut_holds(int first, int last, int slot, int state, int ranges) {
  return state == kCutEmpty || state == kCutWhole ||
         (state == kCutMerge && first >= 0 && first <= last && last < ranges && (slot == 0 || slot == 1));
}

// The tile's place in the flat list, beside the 8 bits of flags of its stage: a
// consumer writes rows for a stage's sequence only if it holds the tile that the
// consumer is at.
PA_HD int tile_tag(int64_t x) { return static_cast<int>(static_cast<uint32_t>(x) << 8); }
PA_HD bool tag_matches(int flags, int64_t x) { return (static_cast<uint32_t>(flags) & ~0xffu) == static_cast<uint32_t>(tile_tag(x)); }

}  // namespace pa
