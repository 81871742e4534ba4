// Limits of the decode kernel's CTAs and the layout of their shared memory, shared by
// the kernel, the host's plan and host-side tests (plain C++ when compiled without nvcc).
#pragma once

#include "pa_schedule.h"

namespace pa {

constexpr int kMaxGroupHeads = 8;  // KV heads per CTA (one consumer warp each)
constexpr int kMaxQueryGroup = 8;  // query heads per KV head (MMA N extent)
constexpr int kMaxColumns = 32;    // (query, head) columns per KV head: four consumer warps of 8
// Producer warps per CTA.  They share the walk over the range's tiles and
// take alternate tiles for the per-tile work (block lookup, stage wait, arm,
// copies), so two tiles' issue latencies overlap.
constexpr int kProducers = 2;
constexpr int kRowSkew = 16;       // fp32 stages: bytes between staged rows beyond the row itself
constexpr uint32_t kLine = 128;    // tensor-core stages: bytes per swizzled line
constexpr int kMaxRowBytes = 2048;  // bytes of one staged token row (K or V)
constexpr int kMaxRanges = 4096;    // bounds the partial-result scratch
constexpr int kFp32Buffers = 9216;  // static shared memory of the fp32 walk with modified scores

struct Layout {
  uint32_t bar, meta, rows, misc, qring, stage, total;
};

// Shared-memory carve-up; identical on host (sizing) and device (addressing).
// Swizzled (tensor-core) stages start on a 1 KiB boundary of the shared
// window, for which `total` keeps 1 KiB of slack.
PA_HD Layout make_layout(int stages, int q_slots, uint32_t q_bytes, uint32_t stage_bytes,
                         bool swizzled) {
  Layout L;
  uint32_t o = 0;
  L.bar = o;
  o += 8u * (2u * stages + 2u * q_slots);
  o = (o + 15u) & ~15u;
  L.meta = o;
  o += 32u * stages;
  L.rows = o;  // per stage: pool row of each tile row holding a new token
  o += 4u * kTile * stages;
  L.misc = o;
  o += 4u * 80u;
  o = (o + 127u) & ~127u;
  L.qring = o;
  o += q_slots * ((q_bytes + 127u) & ~127u);
  o = (o + 127u) & ~127u;
  L.stage = o;
  o += stages * stage_bytes + (swizzled ? 1024u : 0u);
  L.total = o;
  return L;
}

}  // namespace pa
