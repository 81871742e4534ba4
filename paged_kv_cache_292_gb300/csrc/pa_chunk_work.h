// Work decomposition of chunk attention, shared by the kernel, the join and
// host-side tests (plain C++ when compiled without nvcc).
//
// A row tile holds the (token, group head) rows of `tile_tokens` = 128 / group
// (fp32: 64 / group) new tokens of one sequence and KV head, a pair two of them.  An item is one
// sequence, KV head and pair; it walks the tiles of 128 tokens that the pair's
// last row sees.  A tile of an item with two row tiles costs two units, one
// of an item with a single row tile (a chunk's last pair, where its tokens do not
// fill it) one.  All items' units (sequence, head, pair, tile) form one list, cut
// into equal ranges of two units or more, one per CTA; a tile belongs to the range
// of its first unit.  So every CTA gets the same work whatever the batch.  A
// range cuts at most two items: the one that it begins in (partial slot 0) and the one
// that it ends in (slot 1).
#pragma once

#include "pa_schedule.h"

namespace pa {

constexpr int kChunkRows = 128;    // query rows per tile (M of the products)
constexpr int kChunkTokens = 128;  // tokens per tile
constexpr int kChunkRowsF32 = 64;  // query rows per tile over fp32 pools

// sum over i = 0 .. n - 1 of floor((a * i + b) / m), for a, b >= 0, m > 0: the
// quotients of a and b leave a sum over a smaller triangle, whose axes then change
// places (Euclid's steps; Graham, Knuth, Patashnik, Concrete Mathematics, 3.5).
PA_HD int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
  int64_t sum = 0;
  while (n > 0) {
    sum += n * (n - 1) / 2 * (a / m) + n * (b / m);
    a %= m;
    b %= m;
    const int64_t top = a * n + b;
    n = top / m;
    b = top % m;
    const int64_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// A sequence's chunk: n new tokens behind `old` others (negative: the first -old
// of the n have no position and see nothing).
struct ChunkSeq {
  int n, old, tile_tokens;

  PA_HD static int smaller(int a, int b) { return a < b ? a : b; }
  PA_HD int pairs() const { return (n + 2 * tile_tokens - 1) / (2 * tile_tokens); }
  // Tiles that the first `tokens` new tokens see (one at least, whose rows may see nothing).
  PA_HD int tiles_for(int tokens) const {
    const int keys = old + smaller(n, tokens);
    return keys > kChunkTokens ? (keys + kChunkTokens - 1) / kChunkTokens : 1;
  }
  PA_HD int tiles(int pair) const { return tiles_for((pair + 1) * 2 * tile_tokens); }
  // Tiles of the pair's first row tile.
  PA_HD int tiles_first(int pair) const { return tiles_for((2 * pair + 1) * tile_tokens); }
  PA_HD int weight(int pair) const { return n - 2 * pair * tile_tokens > tile_tokens ? 2 : 1; }
  // Units of the pairs before `pair` (0 .. pairs()) of one head.
  PA_HD int64_t before(int pair) const {
    const int full = smaller(pair, pairs() - 1);  // pairs that the chunk fills
    int64_t units = 0;
    if (full > 0) {
      const int64_t step = 2 * tile_tokens;
      int64_t ones = (int64_t)kChunkTokens - old;  // pairs of one tile come first
      ones = ones < step ? 0 : ones / step;
      if (ones > full) ones = full;
      units = 2 * (ones + floor_sum(full - ones, kChunkTokens, step, old + (ones + 1) * step + kChunkTokens - 1));
    }
    if (pair > full) units += (int64_t)tiles(pair - 1) * weight(pair - 1);
    return units;
  }
  PA_HD int64_t units() const { return n > 0 ? before(pairs()) : 0; }
};

// First tile of an item that begins at unit 0 whose first unit is at or behind `unit`.
PA_HD int chunk_tile_at(int64_t unit, int weight, int tiles) {
  if (unit <= 0) return 0;
  const int64_t t = weight == 2 ? (unit + 1) / 2 : unit;
  return t < tiles ? (int)t : tiles;
}

// Ranges for a list of `total` units: two units at least, so that each holds a
// tile's first unit.
PA_HD int chunk_ranges(int64_t total, int most, int least_units) {
  const int64_t r = total / least_units;
  return r < 1 ? 1 : r < most ? (int)r : most;
}

}  // namespace pa
