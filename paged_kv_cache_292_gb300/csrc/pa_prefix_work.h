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

// Units are counted in 32 bits (the host refuses longer lists): the kernel's warps
// work their segments out before their first load, and wide divisions are slow.
struct PrefixWork {
  int tiles;        // prefix tiles
  int pairs;        // row-tile pairs per KV head
  int last_weight;  // units per tile of the last pair: 2, or 1 with a single row tile
  int kv_heads;
  int ctas;

  PA_HD int items() const { return pairs * kv_heads; }
  PA_HD int weight(int item) const { return item % pairs == pairs - 1 ? last_weight : 2; }
  PA_HD uint32_t per_head() const { return (uint32_t)tiles * (2 * (pairs - 1) + last_weight); }
  PA_HD uint32_t total() const { return per_head() * kv_heads; }
  PA_HD uint32_t item_start(int item) const {
    const int head = item / pairs;
    return head * per_head() + (uint32_t)(item - head * pairs) * 2 * tiles;
  }
  PA_HD uint32_t cta_start(int cta) const { return (uint32_t)range_start(cta, total(), ctas); }
  PA_HD int item_of(uint32_t unit) const {
    const uint32_t head = unit / per_head(), pair = (unit - head * per_head()) / (2u * tiles);
    return (int)(head * pairs + (pair < (uint32_t)(pairs - 1) ? pair : pairs - 1));
  }
  // First tile of the item whose first unit is at or behind `unit`.
  PA_HD int tile_at(int item, uint32_t unit) const {
    const uint32_t start = item_start(item);
    if (unit <= start) return 0;
    const uint32_t d = unit - start, t = weight(item) == 2 ? (d + 1) / 2 : d;
    return (int)(t < (uint32_t)tiles ? t : tiles);
  }
  PA_HD int cta_of(int item, int tile) const {  // (for the host check of the list)
    return (int)range_of_tile(item_start(item) + (uint32_t)tile * weight(item), total(), ctas);
  }
  PA_HD int slots() const { return ctas + items(); }
};

// ctas == 0: a list too long for 32-bit units.
PA_HD PrefixWork make_prefix_work(int64_t rows, int kv_heads, int prefix_tokens, int max_ctas) {
  PrefixWork w;
  w.tiles = (prefix_tokens + kPrefixTokens - 1) / kPrefixTokens;
  const int64_t pairs = (rows + 2 * kPrefixRows - 1) / (2 * kPrefixRows);
  w.pairs = (int)pairs;
  w.last_weight = rows - (pairs - 1) * 2 * kPrefixRows > kPrefixRows ? 2 : 1;
  w.kv_heads = kv_heads;
  const int64_t most = (int64_t)w.tiles * (2 * (pairs - 1) + w.last_weight) * kv_heads / 2;
  // Two units at least, so that every range holds a tile's first unit.
  w.ctas = most >= (int64_t(1) << 30) ? 0 : most <= 1 ? 1 : (int)(most < max_ctas ? most : max_ctas);
  return w;
}

}  // namespace pa
