// Host check of the shared-prefix work decomposition in pa_prefix_work.h: every
// tile of every item belongs to exactly one CTA, a CTA's segments have slots of
// their own below slots(), and the join's range of CTAs holds every segment.
#include <stdio.h>

#include <map>
#include <set>
#include <vector>

#include "pa_prefix_work.h"

static int check(int64_t rows, int kv_heads, int prefix, int max_ctas, int take) {
  pa::PrefixWork w = pa::make_prefix_work(rows, kv_heads, prefix, max_ctas);
  if (take < w.ctas) w.ctas = take;  // the kernel may take fewer
  if (w.ctas < 1 || w.ctas > max_ctas) return 1;
  if ((int64_t)w.tiles * 128 < prefix || (int64_t)(w.tiles - 1) * 128 >= prefix) return 2;
  if ((int64_t)w.pairs * 256 < rows || (int64_t)(w.pairs - 1) * 256 >= rows) return 3;
  const int64_t last = rows - (int64_t)(w.pairs - 1) * 256;
  if ((last > 128 ? 2 : 1) != w.last_weight) return 4;
  std::vector<int> owner((size_t)w.items() * w.tiles, -1);
  std::set<int> slots;
  std::map<int, std::set<int>> segments;  // item -> CTAs
  uint32_t before = 0;
  for (int c = 0; c < w.ctas; ++c) {
    const uint32_t a = w.cta_start(c), b = w.cta_start(c + 1);
    if (a != before) return 5;
    before = b;
    const int first = w.item_of(a);
    if (first > 0 && w.item_start(first) > a) return 6;
    for (int i = first; i < w.items() && w.item_start(i) < b; ++i) {
      const int t0 = w.tile_at(i, a), t1 = w.tile_at(i, b);
      if (t0 >= t1) continue;
      if (!slots.insert(c + i).second || c + i >= w.slots()) return 7;
      segments[i].insert(c);
      for (int t = t0; t < t1; ++t) {
        if (owner[(size_t)i * w.tiles + t] != -1) return 8;
        owner[(size_t)i * w.tiles + t] = c;
        if (w.cta_of(i, t) != c) return 9;
      }
    }
  }
  if (before != w.total()) return 10;
  for (int o : owner)
    if (o < 0) return 11;
  for (int i = 0; i < w.items(); ++i) {
    const int c0 = w.cta_of(i, 0), c1 = w.cta_of(i, w.tiles - 1);
    for (int c : segments[i])
      if (c < c0 || c > c1) return 12;
    // The join takes every CTA between the two.
    for (int c = c0; c <= c1; ++c) {
      if (segments[i].count(c) == 0) return 13;
    }
  }
  return 0;
}

int main() {
  // Lists too long for 32-bit units are told apart.
  if (pa::make_prefix_work(1 << 24, 8, 1 << 20, 152).ctas != 0) return 1;
  if (pa::make_prefix_work(1 << 16, 8, 1 << 20, 152).ctas != 152) return 1;
  for (int64_t rows : {1, 5, 127, 128, 129, 255, 256, 257, 384, 385, 640, 1024, 4001})
    for (int heads : {1, 2, 3, 8, 16})
      for (int prefix : {8, 120, 128, 136, 1000, 4096, 20000})
        for (int ctas : {1, 2, 7, 97, 152}) {
          const int rc = check(rows, heads, prefix, 152, ctas);
          if (rc) {
            printf("rows %lld heads %d prefix %d ctas %d: %d\n", (long long)rows, heads, prefix, ctas, rc);
            return 1;
          }
        }
  printf("ok\n");
  return 0;
}
