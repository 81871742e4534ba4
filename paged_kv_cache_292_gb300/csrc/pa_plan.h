// The launch plan of the decode kernel: KV heads per CTA, ranges, the ring of stages in
// shared memory, and the scratch they need.  Host code, shared with host-side tests.
#pragma once

#include "../../include/pagedattn.h"
#include "pa_internal.h"
#include "pa_layout.h"

namespace pa {

struct Plan {
  int Hg, HG, R, stages, q_slots, split, producers;
  int per_sm;  // CTAs per SM
  uint32_t row_bytes, pitch, q_bytes, stage_bytes, smem;
  uint32_t lines, box_rows, box_bytes;  // tensor-core paths (see DecodeParams)
  size_t ws_ml, ws_o, ws_partials;  // places of the partials behind their start, and their bytes
  size_t ws_tickets;                // bytes of the merge tickets
  size_t ws_late;                   // where in a caller's buffer they are if kTicketRoom does not hold them (else 0)
  size_t ws_total;                  // bytes of a caller's buffer
};

// The batch's shape as far as a plan depends on it.  elt: bytes of a pool element;
// q_elt: of a query element (bf16 queries select the tensor-core consumers, whose
// stages are swizzled tensor boxes).
struct PlanShape {
  int num_heads, num_kv_heads, head_size, num_queries, elt, q_elt, block_size;
  bool scaled = false;  // stages hold the tokens' scales, too (int8 pools)

  int group() const { return num_heads / num_kv_heads; }
  int columns() const { return group() * num_queries; }
  bool mma() const { return q_elt == 2; }
};

// A caller's buffer: the merge tickets in its first kTicketRoom bytes, then partial (m, l)
// and O.  A ticket belongs to one KV head of the sequence that the end of a range cuts and
// is found by that range, so that a batch has (R - 1) * num_kv_heads of them however
// many sequences there are.  Their place depends on nothing else: whatever shapes share a
// buffer, and whatever size each call gives for it, no partial lies where another call
// has a ticket.  Calls whose scratch may hold anything leave the room alone, too, so that
// one buffer serves every kind of call.  (By default R * num_kv_heads is at most 8 a CTA:
// 1,216 on 152 SMs.  More tickets than the room holds, where num_ranges is in the hundreds,
// lie behind the call's own partials, and are cleared before its launch.)
// The size is the partials, a ticket for every sequence and KV head, as callers' own formulas have
// it, and of the room what slot 1 of the last range, in which no sequence ends and nothing
// is written, does not pay for: with 4,096 query elements a token and more, nothing.
constexpr size_t kTicketRoom = 16384;

inline size_t workspace_layout(int num_seqs, int num_heads, int num_kv_heads, int head_size, int R, Plan* pl,
                               int num_queries = 1) {
  num_heads *= num_queries;  // partial rows are (query, head) pairs
  const size_t ml = align_up(sizeof(float) * (size_t)R * 2 * num_heads * 2, 256);
  const size_t o = align_up(sizeof(float) * (size_t)R * 2 * num_heads * head_size, 256);
  const size_t cnt = align_up(sizeof(int32_t) * (size_t)num_seqs * num_kv_heads, 256);
  const size_t tickets = align_up(sizeof(int32_t) * (size_t)(R - 1) * num_kv_heads, 256);
  const size_t unused = sizeof(float) * (size_t)num_heads * head_size;  // (a multiple of 256)
  const bool late = tickets > kTicketRoom;
  const size_t total = ml + o + cnt + (kTicketRoom > unused ? kTicketRoom - unused : 0) + (late ? tickets : 0);
  if (pl) {
    pl->ws_ml = 0;
    pl->ws_o = ml;
    pl->ws_partials = ml + o;
    pl->ws_tickets = tickets;
    pl->ws_late = late ? kTicketRoom + ml + o - unused : 0;
    pl->ws_total = total;
  }
  return total;
}

// KV heads one CTA stages per token row: the largest divisor of num_kv_heads
// that is at most `max_heads` (8 with one consumer warp per KV head, 4 with
// two), keeps the row within 2 KiB, so three stages fit in shared memory, and
// makes it whole 128-byte lines (FP8 pools of 64 dims: an even number of heads).
inline int heads_per_cta(int num_kv_heads, int head_size, int elt, int max_heads = kMaxGroupHeads) {
  for (int h = max_heads; h > 1; --h) {
    const int row = h * head_size * elt;
    if (num_kv_heads % h == 0 && row <= kMaxRowBytes && row % (int)kLine == 0) return h;
  }
  return 1;
}

// Consumer warps per KV head: one 8-wide MMA tile of (query, head) columns
// per warp, so ceil(columns / 8) (at most 4: 32 columns).
inline int column_split(int group, int num_queries) { return (group * num_queries + 7) / 8; }

inline int default_ranges(const DeviceInfo& dev, int HG) {
  const int r = dev.sm_count / HG;
  return r < 1 ? 1 : r;
}

inline int gcd_int(int a, int b) {
  while (b != 0) {
    const int t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// The staged rows of CTAs of Hg KV heads.  False: not whole 128-byte lines.
inline bool plan_rows(const PlanShape& s, int Hg, Plan* pl) {
  pl->Hg = Hg;
  pl->HG = s.num_kv_heads / Hg;
  pl->row_bytes = (uint32_t)(Hg * s.head_size * s.elt);
  pl->q_bytes = (uint32_t)(s.num_queries * Hg * s.group() * s.head_size * s.q_elt);
  pl->lines = pl->box_rows = pl->box_bytes = 0;
  if (s.mma()) {
    if (pl->row_bytes % kLine != 0) return false;
    // A tensor copy moves box_rows = gcd(block_size, 16) rows (they share a
    // block) and must land on a 1 KiB boundary under the 128-byte swizzle, so
    // box_rows * lines is a multiple of 8: lines is a multiple of `step`.  An
    // odd multiple spreads consecutive rows over the most bank groups.
    const uint32_t chunks = pl->row_bytes / kLine;
    const int br = gcd_int(s.block_size, kTile);
    const uint32_t step = 8u / (uint32_t)gcd_int(br, 8);
    uint32_t lines = (chunks + step - 1) / step * step;
    if ((lines / step) % 2 == 0) lines += step;
    pl->lines = lines;
    pl->box_rows = (uint32_t)br;
    pl->box_bytes = (uint32_t)br * lines * kLine;
    pl->pitch = lines * kLine;
  } else {
    pl->pitch = pl->row_bytes + kRowSkew;
  }
  pl->stage_bytes = 2u * kTile * pl->pitch;
  if (s.scaled) pl->stage_bytes += (uint32_t)align_up(2 * kTile * sizeof(float) * Hg, 1024);  // (stages start on 1 KiB)
  return true;
}

// The ring of at least `least` stages for `room` bytes of shared memory: the longest,
// where two query slots come before a fourth stage; one slot with four stages only
// where a CTA has the SM to itself (`alone`).
inline bool plan_ring(const PlanShape& s, int room, int least, bool alone, Plan* pl) {
  static const int pref[][2] = {{6, 2}, {5, 2}, {4, 2}, {3, 2}, {3, 1}, {2, 2}, {2, 1}, {4, 1}};  // {stages, query slots}
  for (auto& c : pref) {
    if (!alone && c[0] == 4 && c[1] == 1) continue;
    const Layout L = make_layout(c[0], c[1], pl->q_bytes, pl->stage_bytes, s.mma());
    if ((int)L.total <= room && c[0] >= least) {
      pl->stages = c[0];
      pl->q_slots = c[1];
      pl->smem = L.total;
      return true;
    }
  }
  return false;
}

// Consumers that take two tiles per pass (FP8 pools; bf16 with a KV head's
// columns split over several warps) hold two stages at once: they need four or more.
inline int least_stages(const PlanShape& s) { return s.mma() && (s.elt == 1 || s.columns() > 8) ? 4 : 2; }

// CTAs of the plain walk: one per SM.
inline int plan_plain(const PlanShape& s, const DeviceInfo& dev, Plan* pl) {
  pl->split = column_split(s.group(), s.num_queries);
  pl->producers = kProducers;
  pl->per_sm = 1;
  if (!plan_rows(s, heads_per_cta(s.num_kv_heads, s.head_size, s.elt, kMaxGroupHeads / pl->split), pl))
    return fail(PA_ERR_UNSUPPORTED, "pa_decode: %d KV heads x %d dims make %u-byte rows, not whole 128-byte lines",
                pl->Hg, s.head_size, pl->row_bytes);
  if (!plan_ring(s, dev.max_smem_optin, least_stages(s), true, pl))
    return fail(PA_ERR_UNSUPPORTED, "pa_decode: %d stages of %u bytes do not fit in %d bytes of shared memory",
                least_stages(s), pl->stage_bytes, dev.max_smem_optin);
  return PA_OK;
}

// CTAs of the other walks: of the numbers of KV heads per CTA the one whose consumer
// warps fill an SM's registers best (12 warps fit at 168 a thread, 16 at 128: max_threads),
// among equals the most KV heads (the longest copies); rows of 2 KiB with up to 8
// columns per KV head are HBM-bound as they are and go first.  Then as many of these
// CTAs per SM as the rings of stages leave room for (several keep four stages each,
// fp32 three), which for 128 dims is often one: 4 heads in bf16 run as one CTA of 4
// consumers.  A number of heads whose ring does not fit gives way to the next best.
// One producer warp for few consumers: every warp of the other kind hides latency.
// (96 sequences x 3 queries of 6 x 64 dims: three CTAs per SM 66 us, one 162.)
inline int plan_walk(const PlanShape& s, const DeviceInfo& dev, Plan* pl) {
  const int columns = s.columns();
  const int split = !s.mma() || columns <= 8 ? 1 : (columns + 15) / 16;
  const int warps = s.mma() && (s.head_size == 64 || columns <= 8) ? 16 : 12;
  int below = 1 << 30;  // ranks at or above it have been tried
  for (;;) {
    int best = 0, rank = 0, wanted = 0;
    for (int hg = 1; hg * split <= kMaxGroupHeads; ++hg) {
      const int row = hg * s.head_size * s.elt, consumers = hg * split;
      // Consumers that take two tiles a pass need a ring of four: rows of at most 1 KiB.
      const int most_row = s.mma() && columns > 8 ? kMaxRowBytes / 2 : kMaxRowBytes;
      if (s.num_kv_heads % hg != 0 || row > most_row || (s.mma() && row % (int)kLine != 0)) continue;
      const bool long_rows = row == kMaxRowBytes && columns <= 8;
      int per_sm = long_rows ? 1 : warps / (consumers + (consumers >= 6 ? kProducers : 1));
      if (per_sm < 1) per_sm = 1;
      const int r = 16 * (long_rows ? 100 : consumers * per_sm) + hg;
      if (r < below && r > rank) best = hg, rank = r, wanted = per_sm;
    }
    if (best == 0)
      return fail(PA_ERR_UNSUPPORTED, "pa_decode: no stages of %d KV heads x %d dims fit in %d bytes of shared memory",
                  s.num_kv_heads, s.head_size, dev.max_smem_optin);
    below = rank;
    Plan p{};
    plan_rows(s, best, &p);
    p.split = split;
    p.producers = best * split >= 6 || rank >= 1600 ? kProducers : 1;
    for (int per_sm = wanted; per_sm > 0; --per_sm) {
      // An SM has 228 KiB, of which each of its CTAs takes 1 KiB besides its own.
      const int fixed = s.mma() ? 0 : kFp32Buffers;  // the fp32 consumers' static buffers
      const int room = (per_sm > 1 ? (228 << 10) / per_sm - 1024 : dev.max_smem_optin) - fixed;
      if (plan_ring(s, room, per_sm > 1 ? (s.mma() ? 4 : 3) : least_stages(s), per_sm == 1, &p)) {
        p.per_sm = per_sm;
        *pl = p;
        return PA_OK;
      }
    }
  }
}

// walk: of the walks other than kWalkAll.
inline int make_plan(const PlanShape& s, int num_seqs, int num_ranges, const DeviceInfo& dev, bool walk, Plan* pl) {
  const int rc = walk ? plan_walk(s, dev, pl) : plan_plain(s, dev, pl);
  if (rc != PA_OK) return rc;
  pl->R = num_ranges > 0 ? num_ranges : default_ranges(dev, pl->HG) * pl->per_sm;
  workspace_layout(num_seqs, s.num_heads, s.num_kv_heads, s.head_size, pl->R, pl, s.num_queries);
  return PA_OK;
}

// Scratch of a walk other than kWalkAll over R ranges: the partials, then the cuts.
inline size_t walk_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_size, int R, int num_queries) {
  Plan pl{};
  workspace_layout(num_seqs, num_heads, num_kv_heads, head_size, R, &pl, num_queries);
  return pl.ws_partials + 4 * sizeof(int32_t) * (size_t)num_seqs;
}

// The same for the default number of ranges, whatever the block size (`any_block`: also
// those that are not multiples of 8).  0: no plan.
inline size_t walk_workspace(PlanShape s, int num_seqs, const DeviceInfo& dev, bool any_block) {
  size_t most = 0;
  for (int block = kTile; block >= (any_block ? 1 : kTile); block /= 2) {
    if (block == 8) continue;  // staged like 16
    s.block_size = block;
    Plan pl{};
    if (make_plan(s, num_seqs, 0, dev, true, &pl) != PA_OK) continue;
    const size_t need =
        walk_bytes(num_seqs, s.num_heads, s.num_kv_heads, s.head_size, pl.R, s.num_queries);
    if (need > most) most = need;
  }
  return most;
}

}  // namespace pa
