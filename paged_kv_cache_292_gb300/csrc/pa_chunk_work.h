// Work decomposition of chunk attention, shared by the kernel, the join and
// host-side tests (plain C++ when compiled without nvcc).
//
// A row tile holds the (token, group head) rows of `tile_tokens` = 128 / group
// (fp32: 64 / group) new tokens of one sequence and KV head, a pair two of them.  An item is one
// sequence, KV head and pair; it walks the tiles of 128 tokens that the pair's
// last row sees, a unit of work each (an item whose second row tile is empty takes
// nearly as long: its tiles wait for their copies), and has a few units more for what it
// costs besides.  All items' units (sequence, head, pair, tile) form one list, cut
// into equal ranges, one per CTA; a tile belongs to the range of its unit.  So
// every CTA gets the same work whatever the batch.  A range cuts at most two items:
// the one that it begins in (partial slot 0) and the one that it ends in (slot 1).
#pragma once

#include "pa_schedule.h"

namespace pa {

constexpr int kChunkRows = 128;    // query rows per tile (M of the products)
constexpr int kChunkTokens = 128;  // tokens per tile
// What an item costs besides its tiles (queries in, pipeline up and down, rows out), in tiles:
// about 10,000 clocks to 3,000; fp32: a few to 16,000.
constexpr int kItemUnits = 3, kItemUnitsF32 = 1;
constexpr int kChunkRowsF32 = 64;  // query rows per tile over fp32 pools

// sum over i = 0 .. n - 1 of floor((a * i + b) / 128), for a, b >= 0, n < 2^24: the
// quotients of a and b leave a sum over a smaller triangle, whose axes then change
// places (Euclid's steps; Graham, Knuth, Patashnik, Concrete Mathematics, 3.5).
PA_HD int64_t floor_sum_128(int64_t n, int64_t a, int64_t b) {
  int64_t sum = n * (n - 1) / 2 * (a >> 7) + n * (b >> 7);
  uint32_t x = (uint32_t)a & 127u, m = 128u, y = (uint32_t)b & 127u, k = (uint32_t)n;
  while (x != 0u && k != 0u) {
    const uint32_t top = x * k + y;  // below 2^31
    k = top / m;
    y = top % m;
    const uint32_t t = m;
    m = x;
    x = t;
    sum += (int64_t)k * (k - 1) / 2 * (x / m) + (int64_t)k * (y / m);
    x %= m;
    y %= m;
  }
  return sum;
}

// A sequence's chunk: n new tokens behind `old` others (negative: the first -old
// of the n have no position and see nothing).
struct ChunkSeq {
  int n, old, tile_tokens;
  int item;  // units of an item besides its tiles (kItemUnits)

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
  PA_HD bool two(int pair) const { return n - 2 * pair * tile_tokens > tile_tokens; }  // row tiles
  PA_HD int64_t item_units(int pair) const { return item + tiles(pair); }
  // Units of the pairs before `pair` (0 .. pairs()) of one head.
  PA_HD int64_t before(int pair) const {
    const int full = smaller(pair, pairs() - 1);  // pairs that the chunk fills
    int64_t units = 0;
    if (full > 0) {
      const int64_t step = 2 * tile_tokens;
      int64_t ones = (int64_t)kChunkTokens - old;  // pairs of one tile come first
      ones = ones < step ? 0 : ones / step;
      if (ones > full) ones = full;
      units = (int64_t)full * item + (ones + floor_sum_128(full - ones, step, old + (ones + 1) * step + kChunkTokens - 1));
    }
    if (pair > full) units += item_units(pair - 1);
    return units;
  }
  PA_HD int64_t units() const { return n > 0 ? before(pairs()) : 0; }
};

// First tile at or behind `unit` of an item that begins at unit 0 (the item's own units
// go before its first tile's, which belongs to the item's first unit).
PA_HD int chunk_tile_at(int64_t unit, int tiles, int item) {
  if (unit <= 0) return 0;
  const int64_t t = unit - item;
  return t < 1 ? 1 : t < tiles ? (int)t : tiles;
}

// Ranges for a list of `total` units: so long that each holds a tile's first unit.
PA_HD int chunk_ranges(int64_t total, int most, int item) {
  const int64_t r = total / (item + (item > 1 ? 2 : 1));
  return r < 1 ? 1 : r < most ? (int)r : most;
}

}  // namespace pa
