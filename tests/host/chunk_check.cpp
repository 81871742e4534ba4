// Host check of the chunk work decomposition in pa_chunk_work.h: the closed form of a
// sequence's units, every tile of every item in exactly one range, at most one
// item cut at either end of a range, and the parts that the join adds.
#include <stdio.h>

#include <random>
#include <vector>

#include "pa_chunk_work.h"

struct Item {
  int seq, head, pair, tiles;
  int64_t start;
};

static int64_t slow_units(const pa::ChunkSeq& c, int pairs) {
  int64_t u = 0;
  for (int j = 0; j < pairs; ++j) {
    const int last = (j + 1) * 2 * c.tile_tokens < c.n ? (j + 1) * 2 * c.tile_tokens : c.n;
    const int keys = c.old + last;
    const int tiles = keys <= 128 ? 1 : (keys + 127) / 128;
    u += c.item + tiles;
  }
  return u;
}

static int check(const std::vector<pa::ChunkSeq>& seqs, int heads, int most) {
  const int item_units = seqs[0].item;
  std::vector<Item> items;
  int64_t total = 0;
  for (int s = 0; s < (int)seqs.size(); ++s) {
    const pa::ChunkSeq& c = seqs[s];
    if (c.n == 0) {
      if (c.units() != 0) return 1;
      continue;
    }
    for (int j = 0; j <= c.pairs(); ++j)
      if (c.before(j) != slow_units(c, j)) return 2;
    if (c.units() != c.before(c.pairs())) return 3;
    for (int h = 0; h < heads; ++h)
      for (int j = 0; j < c.pairs(); ++j) {
        items.push_back({s, h, j, c.tiles(j), total});
        total += c.item_units(j);
        if (c.tiles_first(j) > c.tiles(j)) return 4;
      }
  }
  if (total == 0) return 0;
  const int ranges = pa::chunk_ranges(total, most, item_units);
  if (ranges < 1 || ranges > most || (ranges > 1 && total / ranges < item_units + 1)) return 5;
  std::vector<int> first_tile(ranges, 0), first_item(ranges, -1);
  std::vector<std::vector<int>> owner(items.size());
  for (size_t i = 0; i < items.size(); ++i) owner[i].assign(items[i].tiles, -1);
  for (int r = 0; r < ranges; ++r) {
    const int64_t a = pa::range_start(r, total, ranges), b = pa::range_start(r + 1, total, ranges);
    int cut_begin = 0, cut_end = 0;
    for (size_t i = 0; i < items.size(); ++i) {
      const Item& it = items[i];
      const int64_t end = it.start + item_units + it.tiles;
      if (end <= a || it.start >= b) continue;
      const int t0 = pa::chunk_tile_at(a - it.start, it.tiles, item_units);
      const int t1 = pa::chunk_tile_at(b - it.start, it.tiles, item_units);
      if (first_item[r] < 0) {
        first_item[r] = (int)i;
        first_tile[r] = t0 < it.tiles ? t0 : 0;
      }
      if (t0 >= t1) continue;
      for (int t = t0; t < t1; ++t) {
        if (owner[i][t] != -1) return 6;
        owner[i][t] = r;
      }
      if (t0 > 0)
        ++cut_begin;
      else if (t1 < it.tiles)
        ++cut_end;
    }
    if (cut_begin > 1 || cut_end > 1) return 7;
  }
  for (size_t i = 0; i < items.size(); ++i) {
    for (int o : owner[i])
      if (o < 0) return 8;
    // The join: the first range that begins inside the item, the one before it, and those behind.
    int b = -1, last = -1;
    for (int r = 1; r < ranges; ++r)
      if (first_item[r] == (int)i && first_tile[r] > 0) {
        if (b < 0) b = r;
        if (last >= 0 && r != last + 1) return 9;
        last = r;
      }
    const int c0 = owner[i].front(), c1 = owner[i].back();
    if (b < 0 ? c0 != c1 : (c0 != b - 1 || c1 != last)) return 10;
    for (int t = 1; t < items[i].tiles; ++t)
      if (owner[i][t] != owner[i][t - 1] && owner[i][t] != owner[i][t - 1] + 1) return 11;
  }
  return 0;
}

int main() {
  std::mt19937 rng(7);
  auto upto = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int trial = 0; trial < 1500; ++trial) {
    const int group = upto(1, 8), rows = rng() % 4 ? 128 : 64, heads = upto(1, 8);
    std::vector<pa::ChunkSeq> seqs(upto(1, trial % 3 ? 6 : 40));
    const int top = trial % 5 == 0 ? 3000 : trial % 5 == 1 ? 1 : 300, ctx = trial % 7 == 0 ? 40000 : 500;
    for (auto& c : seqs) {
      c.n = rng() % 6 ? upto(1, top) : 0;
      const int context = rng() % 5 ? c.n + upto(0, ctx) : upto(0, c.n);
      c.old = context - c.n;
      c.tile_tokens = rows / group;
      c.item = trial % 4 == 3 ? 0 : trial % 2 ? pa::kItemUnitsF32 : pa::kItemUnits;
    }
    const int rc = check(seqs, heads, rng() % 2 ? 152 : upto(1, 400));
    if (rc) {
      printf("trial %d: %d\n", trial, rc);
      return 1;
    }
  }
  // Long lists.
  pa::ChunkSeq c{1 << 20, 1 << 20, 16, pa::kItemUnits};
  if (c.units() != slow_units(c, c.pairs())) return 1;
  printf("ok\n");
  return 0;
}
