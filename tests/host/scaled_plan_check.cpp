// Host check of the decode kernel's plans over int8 pools, whose stages hold the tokens'
// scales behind K and V (pa_plan.h): no shape that pa_decode_int8 gives to the decode kernel is
// refused, the scales lie inside their stage, and the ring fits.
#include <stdio.h>

#include <initializer_list>

#include "pa_plan.h"

namespace pa {
int fail(int code, const char*, ...) { return code; }
}  // namespace pa

using namespace pa;

static int check(const PlanShape& s) {
  const DeviceInfo dev{0, 152, 232448};
  Plan p{};
  if (make_plan(s, 100, 0, dev, false, &p) != PA_OK) return 1;
  const Layout L = make_layout(p.stages, p.q_slots, p.q_bytes, p.stage_bytes, true);
  if (L.total != p.smem || (int)L.total > dev.max_smem_optin) return 2;
  if (p.stages < least_stages(s) || p.stages < 4) return 3;  // a pass takes two
  if (p.stage_bytes % 1024 != 0) return 4;
  // K, V, then [K, V][head][16] floats.
  const uint32_t scales = 2u * kTile * p.lines * kLine;
  if (scales % 16 != 0 || scales + 2u * p.Hg * kTile * 4u > p.stage_bytes) return 5;
  if (p.Hg * p.HG != s.num_kv_heads || p.row_bytes % kLine != 0 || p.lines * kLine < p.row_bytes) return 6;
  if (p.split * 8 < s.columns() || p.Hg * p.split > kMaxGroupHeads) return 7;
  if (p.ws_late != 0) return 8;
  return 0;
}

int main() {
  int plans = 0;
  for (int D : {64, 128})
    for (int Hk = 1; Hk <= 64; ++Hk)
      for (int G = 1; G <= kMaxQueryGroup; ++G)
        for (int Q = 1; G * Q <= kMaxColumns; ++Q)
          for (int bs : {1, 2, 3, 4, 6, 8, 12, 16, 24, 40, 4096}) {
            if (Hk * D % (int)kLine != 0) continue;  // these run as chunks
            ++plans;
            const int rc = check(PlanShape{Hk * G, Hk, D, Q, 1, 2, bs, true});
            if (rc) {
              printf("D %d Hk %d G %d Q %d block %d: %d\n", D, Hk, G, Q, bs, rc);
              return 1;
            }
          }
  printf("ok, %d plans\n", plans);
  return 0;
}
