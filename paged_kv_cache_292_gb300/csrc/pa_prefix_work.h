// Work decomposition of the shared-prefix kernel, shared by the kernel, the
// join and host-side tests (plain C++ when compiled without nvcc).
//
// The query rows of one KV head (sequence, query, group head) are cut into
// pairs of 128-row tiles.  An item is one KV head and one pair; it walks all of
// the prefix's tiles of 128 tokens.  A tile of an item with two row tiles costs two
// units, one of an item with a single row tile (the last pair when the rows do
// not fill it) one.  All items' units, item after item, form one list, cut
// into as many equal ranges as there are CTAs; a tile belongs to the range of
// its first unit.  So every CTA gets the same work whatever the batch, and a
// CTA's part of an item (a segment) leaves one partial result in slot
// cta + item, which no other segment has: along the list either number rises.
#pragma once

#include "pa_schedule.h"

namespace pa {

constexpr int kPrefixRows = 128;    // query rows per tile (M of the products)
constexpr int kPrefixTokens = 128;  // tokens per tile

struct PrefixWork {
  int tiles;        // prefix tiles
  int pairs;        // row-tile pairs per KV head
  int last_weight;  // units per tile of the last pair: 2, or 1 with a single row tile
  int kv_heads;
  int ctas;

  PA_HD int items() const { return pairs * kv_heads; }
  PA_HD int weight(int item) const { return item % pairs == pairs - 1 ? last_weight : 2; }
  PA_HD int64_t per_head() const { return (int64_t)tiles * (2 * (pairs - 1) + last_weight); }
  PA_HD int64_t total() const { return per_head() * kv_heads; }
  PA_HD int64_t item_start(int item) const {
    return (item / pairs) * per_head() + (int64_t)(item % pairs) * 2 * tiles;
  }
  PA_HD int64_t cta_start(int cta) const { return range_start(cta, total(), ctas); }
  PA_HD int item_of(int64_t unit) const {
    const int64_t head = unit / per_head(), pair = (unit - head * per_head()) / (2 * (int64_t)tiles);
    return (int)(head * pairs + (pair < pairs - 1 ? pair : pairs - 1));
  }
  // First tile of the item whose first unit is at or behind `unit`.
  PA_HD int tile_at(int item, int64_t unit) const {
    const int64_t d = unit - item_start(item);
    if (d <= 0) return 0;
    const int w = weight(item);
    const int64_t t = (d + w - 1) / w;
    return (int)(t < tiles ? t : tiles);
  }
  PA_HD int cta_of(int item, int tile) const {
    return (int)range_of_tile(item_start(item) + (int64_t)tile * weight(item), total(), ctas);
  }
  PA_HD int slots() const { return ctas + items(); }
};

PA_HD PrefixWork make_prefix_work(int64_t rows, int kv_heads, int prefix_tokens, int max_ctas) {
  PrefixWork w;
  w.tiles = (prefix_tokens + kPrefixTokens - 1) / kPrefixTokens;
  w.pairs = (int)((rows + 2 * kPrefixRows - 1) / (2 * kPrefixRows));
  w.last_weight = rows - (int64_t)(w.pairs - 1) * 2 * kPrefixRows > kPrefixRows ? 2 : 1;
  w.kv_heads = kv_heads;
  // Two units at least, so that every range holds a tile's first unit.
  w.ctas = 1;
  const int64_t most = w.total() / 2;
  if (most > 1) w.ctas = (int)(most < max_ctas ? most : max_ctas);
  return w;
}

}  // namespace pa
