// Host check of the walks in pa_schedule.h, range by range as the decode kernel goes
// through them: every token to attend is in exactly one tile, every partial is
// written once, the cut of a sequence names just the partials that its ranges wrote,
// and the checks that the kernels make before they use a stage or a cut accept all
// of these and refuse what a lost stage or cut would hold.
#include <stdio.h>

#include <set>
#include <utility>
#include <vector>

#include "pa_schedule.h"

static unsigned seed = 4321;
static int rnd(int n) {
  seed = seed * 1103515245u + 12345u;
  return (int)((seed >> 8) % (unsigned)n);
}

struct Seq {
  int c, first, pre;
};

template <int WALK>
static pa::SeqSpan<WALK> span(const Seq& q, int prefix, int queries, int window) {
  pa::SeqSpan<WALK> w;
  if (WALK == pa::kWalkAll) w.all(q.c);
  if (WALK == pa::kWalkRest) w.rest(q.c, prefix, queries);
  if (WALK == pa::kWalkMod) w.seen(q.c, q.first, q.pre, queries, window);
  return w;
}

// Whether some query of the sequence sees token t (the definition).
static bool seen_by_some(const Seq& q, int t, int queries, int window) {
  for (int i = 0; i < queries; ++i) {
    const int pos = q.c - queries + i;
    if (pos < 0 || t >= q.c || t < q.first) continue;
    if (t < q.pre || (t <= pos && pos - t < window)) return true;
  }
  return false;
}

template <int WALK>
static int check(const std::vector<Seq>& seqs, int R, int left, int prefix, int queries, int window) {
  const int S = (int)seqs.size();
  std::vector<int64_t> at(S + 1, 0);
  for (int s = 0; s < S; ++s) at[s + 1] = at[s] + span<WALK>(seqs[s], prefix, queries, window).n;
  const int64_t total = at[S];
  int64_t Reff = total < R ? total : R;
  if (left < Reff) Reff = left;  // a walk beside the prefix kernel takes fewer
  if (total == 0) return 0;
  std::set<std::pair<int64_t, int>> written;      // (range, slot)
  std::vector<std::set<std::pair<int64_t, int>>> parts(S);
  std::vector<int> whole(S, 0);
  std::vector<std::vector<char>> took(S);
  for (int s = 0; s < S; ++s) took[s].assign(seqs[s].c + 64, 0);
  for (int64_t r = 0; r < Reff; ++r) {
    const int64_t a = pa::range_start(r, total, Reff), b = pa::range_start(r + 1, total, Reff);
    if (a >= b) return 1;
    int s = 0;
    while (at[s + 1] <= a) ++s;
    int slot = 0;
    for (int64_t x = a; x < b; ++x) {
      bool begins = x == a;
      while (x >= at[s + 1]) {
        if (++s >= S) return 2;
        begins = true;
      }
      const auto w = span<WALK>(seqs[s], prefix, queries, window);
      if (begins) slot = pa::segment_slot(a, b, at[s], at[s + 1]);
      const int tok0 = w.token((int)(x - at[s]));
      if (tok0 < 0 || tok0 >= w.c) return 3;
      int seen = 0;
      for (int t = tok0; t < tok0 + pa::kTile; ++t) {
        if (WALK == pa::kWalkMod ? !w.sees(t) : t >= w.c) continue;
        if (took[s][t]++) return 4;
        ++seen;
      }
      if (seen == 0) return 5;
      const int flags = ((slot + 1) << 2) | 3 | pa::tile_tag(x);
      if (!pa::tag_matches(flags, x) || ((flags >> 2) & 3) - 1 != slot) return 6;
      for (int off : {1, 2, 3, 4, 5, 6, 12})  // what the stage held before, or holds next
        if (pa::tag_matches(flags, x + off) || pa::tag_matches(flags, x - off)) return 7;
      if (x == b - 1 || x == at[s + 1] - 1) {
        if (slot < 0) {
          ++whole[s];
        } else {
          if (!written.insert({r, slot}).second) return 8;
          parts[s].insert({r, slot});
        }
      }
    }
  }
  for (int s = 0; s < S; ++s) {
    const auto w = span<WALK>(seqs[s], prefix, queries, window);
    for (int t = 0; t < seqs[s].c; ++t) {
      const bool need = WALK == pa::kWalkAll    ? true
                        : WALK == pa::kWalkRest ? t >= w.t0
                                                : seen_by_some(seqs[s], t, queries, window);
      if (need != (took[s][t] != 0)) return 9;
    }
    if (w.n == 0) {
      if (whole[s] || !parts[s].empty()) return 10;
      continue;
    }
    const int r0 = (int)pa::range_of_tile(at[s], total, Reff), r1 = (int)pa::range_of_tile(at[s + 1] - 1, total, Reff);
    const int slot0 = pa::partial_slot_of_range(r0, at[s], total, Reff);
    const int state = r0 == r1 ? pa::kCutWhole : pa::kCutMerge;
    if (!pa::cut_holds(r0, r1, slot0, state, R)) return 11;
    std::set<std::pair<int64_t, int>> named;
    if (state == pa::kCutMerge)
      for (int k = r0; k <= r1; ++k) named.insert({k, k == r0 ? slot0 : 0});
    if (named != parts[s] || whole[s] != (state == pa::kCutWhole)) return 12;
  }
  return 0;
}

int main() {
  using namespace pa;
  for (int bad : {-1, 3, 4, 0x3f800000, -0x40800000})
    if (cut_holds(0, 1, 0, bad, 152)) return 1;
  if (cut_holds(-1, 1, 0, kCutMerge, 152) || cut_holds(0, 152, 0, kCutMerge, 152) || cut_holds(5, 4, 0, kCutMerge, 152) ||
      cut_holds(0, 1, 2, kCutMerge, 152) || cut_holds(0, 1, -1, kCutMerge, 152) ||
      cut_holds(0x7fffffff, (int)0x80000000, 0, kCutMerge, 152))
    return 1;
  if (!cut_holds(0, 151, 1, kCutMerge, 152) || !cut_holds(7, 7, 0, kCutMerge, 152)) return 1;
  if (!tag_matches(tile_tag((int64_t(1) << 40) + 5) | 0x1f, (int64_t(1) << 40) + 5)) return 1;
  for (int trial = 0; trial < 4000; ++trial) {
    const int S = 1 + rnd(trial % 10 == 0 ? 315 : 40), queries = 1 + rnd(8), R = 1 + rnd(320), left = 1 + rnd(R);
    const int block = 8 * (1 + rnd(4)), prefix = block * rnd(40), reach = 1 + rnd(trial % 3 ? 40 : 700);
    const int window = rnd(3) ? 1 + rnd(200) : kNoWindow;
    std::vector<Seq> seqs(S);
    for (Seq& q : seqs) {
      q.c = rnd(10) ? prefix + queries + rnd(reach) : rnd(prefix + queries);
      if (rnd(12) == 0) q.c = 0;
      q.first = rnd(3) ? 0 : rnd(q.c + 20);
      q.pre = rnd(2) ? 0 : rnd(q.c + 20);
      if (rnd(40) == 0) q.first = 0x7fffffff;
      if (rnd(40) == 0) q.pre = 0x7fffffff;
    }
    int rc = check<kWalkRest>(seqs, R, left, prefix, queries, 0);
    if (rc == 0) rc = check<kWalkMod>(seqs, R, R, prefix, queries, window);
    if (rc == 0) rc = check<kWalkAll>(seqs, R, R, prefix, queries, 0);
    if (rc) {
      printf("trial %d S %d queries %d R %d left %d prefix %d window %d: %d\n", trial, S, queries, R, left, prefix,
             window, rc);
      return 1;
    }
  }
  printf("ok\n");
  return 0;
}
