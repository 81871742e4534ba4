// Host check of the decode kernel's launch plans (pa_plan.h) over every batch shape that
// the entry points take: none is refused, CTAs fit the SM as often as the plan says,
// consumers that take two tiles a pass have four stages, and the scratch sizes handed
// out hold the plan's.
#include <stdio.h>

#include <initializer_list>

#include "pa_plan.h"

namespace pa {
int fail(int code, const char*, ...) { return code; }
}  // namespace pa

using namespace pa;
static const DeviceInfo kDev{0, 152, 232448};

static int check(const PlanShape& s, bool walk) {
  Plan p{};
  if (make_plan(s, 100, 0, kDev, walk, &p) != PA_OK) return 1;
  const Layout L = make_layout(p.stages, p.q_slots, p.q_bytes, p.stage_bytes, s.mma());
  const int fixed = walk && !s.mma() ? kFp32Buffers : 0;
  if (L.total != p.smem || (int)L.total + fixed > kDev.max_smem_optin) return 2;
  if (p.per_sm > 1 && p.per_sm * ((int)L.total + fixed + 1024) > 228 << 10) return 3;
  if (p.stages < least_stages(s) || p.Hg * p.HG != s.num_kv_heads) return 4;
  const int consumers = p.Hg * p.split, threads = 32 * (consumers + p.producers);
  if (consumers > kMaxGroupHeads || p.Hg * s.head_size * s.elt > kMaxRowBytes) return 5;
  if (p.split * (s.mma() && walk && s.columns() > 8 ? 16 : 8) < s.columns()) return 6;
  // Registers: 168 a thread, or 128 (max_threads).
  const bool small = walk && s.mma() && (s.head_size == 64 || s.columns() <= 8);
  if (p.per_sm > 1 && p.per_sm * threads > (small ? 512 : 384)) return 7;
  if (s.mma() && (p.box_bytes % 1024 != 0 || p.row_bytes % kLine != 0)) return 8;
  if (p.R < 1 || p.R > kMaxRanges) return 9;
  if (!walk) return 0;
  // The scratch handed out for the walk holds what this block size needs.
  const size_t need = walk_bytes(100, s.num_heads, s.num_kv_heads, s.head_size, p.R, s.num_queries);
  if (walk_workspace(s, 100, kDev, true) < need) return 10;
  if (s.block_size % 8 == 0 && walk_workspace(s, 100, kDev, false) < need) return 11;
  return 0;
}

int main() {
  int plans = 0;
  for (int D : {64, 128})
    for (int Hk = 1; Hk <= 24; ++Hk)
      for (int G = 1; G <= 8; ++G)
        for (int Q = 1; Q == 1 || G * Q <= 32; ++Q)
          for (int bs : {1, 2, 3, 4, 6, 8, 12, 16, 24, 40, 4096})
            for (int kind = 0; kind < 3; ++kind) {  // fp32, bf16, FP8 pools
              if (kind == 0 && Q > 1) continue;
              if (kind == 2 && D == 64 && Hk % 2 != 0) continue;
              const int elt = kind == 0 ? 4 : kind == 1 ? 2 : 1;
              const PlanShape s{Hk * G, Hk, D, Q, elt, kind == 0 ? 4 : 2, bs};
              for (bool walk : {false, true}) {
                ++plans;
                const int rc = check(s, walk);
                if (rc) {
                  printf("elt %d D %d Hk %d G %d Q %d block %d walk %d: %d\n", elt, D, Hk, G, Q, bs, walk, rc);
                  return 1;
                }
              }
            }
  printf("ok, %d plans\n", plans);
  return 0;
}
