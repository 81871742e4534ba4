// Host check of the scratch of decode calls (pa_plan.h): in a buffer that calls of any
// shapes share no partial of one lies where another has a merge ticket, every write stays
// inside the size handed out, and cut sequences of a batch have tickets of their own.
#include <stdio.h>

#include <initializer_list>
#include <set>
#include <vector>

#include "pa_plan.h"

namespace pa {
int fail(int code, const char*, ...) { return code; }
}  // namespace pa

using namespace pa;

static unsigned seed = 77;
static int rnd(int n) {
  seed = seed * 1103515245u + 12345u;
  return (int)((seed >> 8) % (unsigned)n);
}

// The bytes that a call may write as partials, and as tickets.
struct Places {
  size_t part0, part1, ticket0, ticket1, total;
  bool cleared;
};

static Places places(int S, int H, int Hk, int D, int R, int Q) {
  Plan p{};
  Places w{};
  w.total = workspace_layout(S, H, Hk, D, R, &p, Q);
  if (w.total != p.ws_total) w.total = 0;
  const size_t rows = (size_t)H * Q;
  // The last slot that a range ends in: slot 1 of range R - 2, or slot 0 of range R - 1.
  const size_t slots = 2 * (size_t)R - 1;
  w.part0 = kTicketRoom + p.ws_ml;
  w.part1 = kTicketRoom + p.ws_o + slots * rows * D * 4;
  if (kTicketRoom + p.ws_ml + slots * rows * 8 > kTicketRoom + p.ws_o) w.total = 0;
  w.cleared = p.ws_late != 0;
  w.ticket0 = p.ws_late;
  w.ticket1 = w.ticket0 + (size_t)(R - 1) * Hk * 4;
  return w;
}

static int check_layout(const Places& w) {
  if (w.part1 > w.total || w.ticket1 > w.total || w.part0 % 256 != 0 || w.ticket0 % 256 != 0) return 1;
  // Tickets that are not cleared before a launch: where no call has anything else.
  if (!w.cleared && w.ticket1 > kTicketRoom) return 2;
  if (w.part0 < kTicketRoom) return 3;
  // Those that are: away from the call's own partials.
  if (w.cleared && w.ticket0 < w.part1) return 4;
  return 0;
}

// Cut sequences of random batches: r0 is below the last range and no other sequence's, and
// slot 1 of the last range stays unused.
static int check_ranges() {
  for (int trial = 0; trial < 3000; ++trial) {
    const int S = 1 + rnd(60), R = 1 + rnd(200);
    std::vector<int64_t> at(S + 1, 0);
    for (int s = 0; s < S; ++s) at[s + 1] = at[s] + (rnd(8) ? rnd(90) : 0);
    const int64_t total = at[S], Reff = total < R ? total : R;
    std::set<int64_t> taken;
    for (int s = 0; s < S; ++s) {
      if (at[s + 1] == at[s]) continue;
      const int64_t r0 = range_of_tile(at[s], total, Reff), r1 = range_of_tile(at[s + 1] - 1, total, Reff);
      if (r0 == r1) continue;
      if (r0 >= R - 1 || !taken.insert(r0).second) return 5;
      for (int64_t r = r0; r <= r1; ++r)
        if (r == R - 1 && (r == r0 ? partial_slot_of_range(r0, at[s], total, Reff) : 0) != 0) return 6;
    }
  }
  return 0;
}

int main() {
  const DeviceInfo dev{0, 152, 232448};
  int shapes = 0;
  for (int D : {64, 128})
    for (int Hk : {1, 2, 3, 5, 8, 16, 24, 64})
      for (int G : {1, 2, 3, 4, 8})
        for (int Q : {1, 2, 3, 4, 8, 16, 32}) {
          if (G * Q > kMaxColumns) continue;
          for (int S : {1, 2, 4, 7, 64, 300, 1033, 1300, 8192, 1000000})
            for (int R : {0, 1, 2, 3, 7, 152, 400, 513, 514, 700, 4096}) {
              int ranges = R;
              if (R == 0) {  // the default
                PlanShape s{Hk * G, Hk, D, Q, 2, 2, 16};
                Plan p{};
                if (make_plan(s, S, 0, dev, false, &p) != PA_OK) return 1;
                ranges = p.R;
                if (p.ws_late != 0) {
                  printf("default plan without room: Hk %d D %d\n", Hk, D);
                  return 1;
                }
              }
              ++shapes;
              const int rc = check_layout(places(S, Hk * G, Hk, D, ranges, Q));
              if (rc) {
                printf("D %d Hk %d G %d Q %d S %d R %d: %d\n", D, Hk, G, Q, S, ranges, rc);
                return 1;
              }
            }
        }
  const int rc = check_ranges();
  if (rc) {
    printf("ranges: %d\n", rc);
    return 1;
  }
  printf("ok, %d shapes\n", shapes);
  return 0;
}
