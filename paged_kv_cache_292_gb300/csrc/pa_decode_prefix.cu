// Decode attention of a batch that shares a long prefix (pa_decode_prefix).
//
// The softmax over a sequence's tokens splits into the prefix's P tokens and
// the rest.  For the prefix, K and V are the same for all sequences, so the
// (sequence, query, group head) rows of one KV head are the rows of two matrix
// products, S = Q K^T and O = P V, that read the prefix once:
//
//   m_r = max_t s_rt, l_r = sum_t 2^(s_rt - m_r), O_r = sum_t 2^(s_rt - m_r) v_t
//
// (s in log2 units).  The rest is the decode kernel's walk behind the prefix
// (kWalkRest), and the join adds the parts of a row by their maxima.
//
// Prefix kernel: one persistent CTA per SM, equal shares of the (KV head, pair
// of 128-row tiles, 128-token tile) list (pa_prefix_work.h).  Per CTA:
//   warps 0-7, 8-15 softmax groups 0 and 1: two threads per row, 64 tokens each,
//                   which exchange their maxima; scores come from tensor memory,
//                   weights go back there as bf16
//   warp 16         loads K and V tiles by TMA: boxes of gcd(block_size, 128)
//                   token rows x 64 elements, into 128-byte swizzled panels
//                   (FP8 pools: the codes as they are, into a ring of their own)
//   warp 17         issues the products (tcgen05.mma, one thread): S from Q and K in
//                   shared memory, O from the weights in tensor memory and V
//   warps 18, 19    FP8 pools: widen the codes to f16 into the panels; queries and
//                   weights are f16 then, too (2^-11)
// With two row tiles each group has one and both use every K/V tile; with a
// single row tile the groups take alternate K/V tiles and leave a partial
// each.  While one group exponentiates, the tensor core works for the other.
// Tensor memory: S0, S1 (128 columns each; the weights overwrite the first 64,
// their second parts, if any, the other 64), O0, O1 (D columns each).
//
// What bounds it: with two row tiles the products.  A K/V tile pair of two row tiles
// (16.8 MFLOP at D = 128) takes 1.82 us, its four products alone 1.47, and at the rate
// of a large library product (1.88 PFLOP/s over 152 SMs) they would take 1.36; the rest
// is softmax that the tensor core waits for.  With one row tile the copies bound it.
// Around that stand about 25 us: start-up 9, uneven ends 5, the join 3 to 7.  Measured,
// whole calls: 64 sequences on 4k shared tokens 39 us (152 MB, 22 us of HBM time), 9 x 4
// queries on 32k 73 us (39 GFLOP, 21 us), 256 on 16k 203 us (1.14 GB, 168 us: the
// tokens behind the prefix).  One thread per row instead of two: 54 us for 64 on 4k.
// Blocks of 8 tokens take about a quarter longer than blocks of 16 or more (smaller boxes).
// FP8 pools: 64 sequences on 4k 42 us, 256 on 16k with 16 tokens of their own 88 (bf16 83).
#include "pa_launch.cuh"

#include <cmath>
#include <utility>

#include "pa_decode_impl.h"
#include "pa_prefix_work.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kPrefixThreads = 640;
// Registers per thread: 96 at launch (65536 / 640, rounded down); a softmax thread
// holds 64 scores, the fifth warpgroup issues copies and products.
// 4 * 128 * 104 + 128 * 64 = 640 * 96.
constexpr int kSoftmaxRegisters = 104, kIssueRegisters = 64;
constexpr int kSoftmaxWarps = 16, kLoadWarp = 16, kProductWarp = 17, kWidenWarp = 18, kWidenWarps = 2;
constexpr uint32_t kPanel = 128 * 128;  // bytes of 128 rows x 64 bf16
// A running maximum is kept until a tile exceeds it by this factor (log2): until
// then weights are at most 2^8, which bf16 and the fp32 sums hold as well as 1.
constexpr float kSlack = 8.f;
// FP8 pools: the weights are f16, whose upper range they use: up to 2^15 with the slack.
// They keep 11 bits down to 2^-21 of the running maximum's and vanish below 2^-32.
constexpr float kWeightUp = 7.f;

struct PrefixParams {
  CUtensorMap tm_k, tm_v;  // (64 elements, chunk of 64 within a token row, token row); FP8: (D, KV head, token row)
  const __nv_bfloat16* q;
  const int32_t* table;
  int32_t* error_flag;
  float* part_ml;  // [slots][2][128][2]
  float* part_o;   // [slots][2][D / 4][128][4]: a thread's row side by side with its neighbours'
  PrefixWork work;  // `ctas`: at most; what the walk behind the prefix leaves is taken (prefix_share)
  int2* item_ctas;  // [items]: first and last CTA with a partial
  const int32_t* context_lens;
  int num_seqs, num_queries, max_tokens;  // of the walk: its tiles,
  int walk_groups, walk_row_bytes;        // and the shape of its CTAs
  int sm_count;
  int rows;  // query rows per KV head
  int group, num_heads, block_size, prefix_tokens, num_physical_blocks, box_rows;
  // Scores are scale_log2 * <(q & q_keep) ^ q_flip, k>: a negative scale changes the
  // queries' signs and a scale of zero makes them zero, so that scale_log2 > 0
  // and the largest product is the largest score.
  float scale_log2;
  uint32_t q_keep, q_flip;
  unsigned long long wait_limit_ns;
  long long stall_tile;  // tests of the bounded waits: item * tiles + tile whose copies are withheld
};

// Work of the list for prefix_share: its units, and what a segment costs besides
// (queries in, pipeline up and down, partials out), about five units.
__host__ __device__ __forceinline__ float prefix_cost(const PrefixWork& w) {
  return static_cast<float>(w.total()) + 5.f * (w.items() + 0.25f * w.ctas);
}

template <int D, bool F8>
struct PrefixLayout {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kTileBytes = kPanels * kPanel;  // a Q, K or V tile
  static constexpr int kStages = D == 64 ? 8 : F8 ? 3 : 5;
  static constexpr int kRawStages = F8 ? (D == 64 ? 8 : 4) : 0;  // tiles of codes
  static constexpr uint32_t kRawBytes = kTileBytes / 2;
  static constexpr uint32_t kExchange = 1024;  // [2 groups][2 halves][128] floats; barriers before it
  static constexpr uint32_t kQ = 3 * 1024;
  static constexpr uint32_t kRing = kQ + 2 * kTileBytes;
  static constexpr uint32_t kRaw = kRing + kStages * kTileBytes;
  static constexpr uint32_t kBytes = kRaw + kRawStages * kRawBytes;
};

template <int D, bool F8>
__global__ void __launch_bounds__(kPrefixThreads, 1) pa_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using L = PrefixLayout<D, F8>;
  constexpr int NS = L::kStages, NR = L::kRawStages;
  extern __shared__ __align__(1024) unsigned char smem[];  // swizzled panels start on 1 KiB boundaries
  const uint32_t base = smem_addr(smem);
  if ((base & 1023u) != 0) {  // cannot be: the array asks for it
    if (threadIdx.x == 0) report(p.error_flag, PA_DEVERR_TIMEOUT);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t bars = base;
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 8u * (NS + i); };
  const uint32_t q_full = bars + 8u * (2 * NS);
  auto s_full = [&](int w) { return bars + 8u * (2 * NS + 1 + w); };
  auto p_full = [&](int w) { return bars + 8u * (2 * NS + 3 + w); };
  auto o_full = [&](int w) { return bars + 8u * (2 * NS + 5 + w); };
  const uint32_t drained = bars + 8u * (2 * NS + 7);
  auto exchanged = [&](int w) { return bars + 8u * (2 * NS + 8 + w); };
  auto raw_full = [&](int i) { return bars + 8u * (2 * NS + 10 + i); };
  auto raw_empty = [&](int i) { return bars + 8u * (2 * NS + 10 + NR + i); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 512);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + 516);
  auto timed_out = [&]() {
    if (lane == 0) {
      report(p.error_flag, PA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  griddep_wait();
  griddep_launch_dependents();  // the walk behind the prefix runs on the SMs left to it

  // This kernel's share of the SMs, the same in every CTA.
  PrefixWork wk = p.work;
  {
    long long* sums = reinterpret_cast<long long*>(smem + 640);
    long long walk = 0;
    for (int s = tid; s < p.num_seqs; s += kPrefixThreads) {
      const int c = max(0, min(__ldg(p.context_lens + s), p.max_tokens));
      walk += tiles_of(c >= p.prefix_tokens + p.num_queries - 1 ? c - p.prefix_tokens : c);
    }
    walk = warp_sum_ll(walk);
    if (lane == 0) sums[warp] = walk;
    __syncthreads();
    walk = 0;
    for (int i = 0; i < kPrefixThreads / 32; ++i) walk += sums[i];
    wk.ctas = min(wk.ctas, prefix_share(prefix_cost(wk), walk, p.num_seqs, p.walk_groups,
                                        walk_tile_us(p.walk_row_bytes, p.group * p.num_queries),
                                        p.num_queries * p.num_heads * D, D, p.sm_count));
  }
  const int cta = blockIdx.x;
  if (cta >= wk.ctas) return;
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), F8 ? kWidenWarps : 1);
      mbar_init(empty(i), 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), kWidenWarps);
    }
    mbar_init(q_full, kSoftmaxWarps);
    for (int w = 0; w < 2; ++w) {
      mbar_init(exchanged(w), kSoftmaxWarps / 2);
      mbar_init(s_full(w), 1);
      mbar_init(p_full(w), kSoftmaxWarps / 2);
      mbar_init(o_full(w), 1);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == kProductWarp) tmem_alloc(smem_addr(smem + 516), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t ua = wk.cta_start(cta), ub = wk.cta_start(cta + 1);
  const int first_item = wk.item_of(ua);
  // Weights in two bf16 parts where one row tile is all: 32 sequences on 8k 31.2 -> 33.2
  // us; with two row tiles the further products would cost 9x4 queries on 32k 74 -> 87.
  const bool fine = !F8 && wk.pairs == 1 && wk.last_weight == 1;

  if (warp < kSoftmaxWarps)
    registers_up<kSoftmaxRegisters>();
  else
    registers_down<kIssueRegisters>();

  if (warp < kSoftmaxWarps) {
    // ---------------- softmax ----------------
    const int w = warp >> 3, half = (warp >> 2) & 1, row = tid & 127;
    constexpr float kUp = F8 ? kWeightUp : 0.f;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the TMEM lanes
    const uint32_t s_addr = tmem + lanes + 128u * w, o_addr = tmem + lanes + 256u + (uint32_t)D * w + (D / 2) * half;
    float* mine = reinterpret_cast<float*>(smem + L::kExchange) + (w * 2 + half) * 128 + row;
    const float* other = reinterpret_cast<const float*>(smem + L::kExchange) + (w * 2 + (half ^ 1)) * 128 + row;
    uint32_t s_phase = 0, o_phase = 0, x_phase = 0;
    // Give the row's other thread `v` and get its value.  (What it gave before has
    // been read: either the weights of the tile in between, which the tensor core
    // waits for, or the next queries came after that.)
    auto exchange = [&](float v, float* got) -> bool {
      *mine = v;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(exchanged(w));
      if (!wait_or_abort(exchanged(w), x_phase, p.wait_limit_ns, abort_flag)) return false;
      x_phase ^= 1u;
      tc_fence_after();
      *got = *other;
      return true;
    };
    for (int item = first_item; item < wk.items() && wk.item_start(item) < ub; ++item) {
      const int t0 = wk.tile_at(item, ua), t1 = wk.tile_at(item, ub);
      if (t0 >= t1) continue;
      const bool two = wk.weight(item) == 2;
      const int head = item / wk.pairs, row0 = (item % wk.pairs) * 2 * kPrefixRows;
      // The row's queries into the swizzled Q tile: half a row per thread with
      // two row tiles, a quarter with one.
      {
        const int r = row0 + (two ? w * kPrefixRows : 0) + row;
        constexpr int kUnits = D / 8;  // 16-byte units of a row
        const int n = two ? kUnits / 2 : kUnits / 4, u0 = n * (two ? half : 2 * w + half);
        const uint4* src = nullptr;
        if (r < p.rows) {
          const int tok = r / p.group, g = r - tok * p.group;
          src = reinterpret_cast<const uint4*>(p.q + ((size_t)tok * p.num_heads + head * p.group + g) * D);
        }
        unsigned char* dst = smem + L::kQ + (two ? w * L::kTileBytes : 0) + row * 128;
        uint4 v[kUnits / 2];
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i)
          v[i] = src != nullptr && i < n ? __ldg(src + u0 + i) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i) {
          if (i < n) {
            const int u = u0 + i;
            v[i].x = (v[i].x & p.q_keep) ^ p.q_flip;
            v[i].y = (v[i].y & p.q_keep) ^ p.q_flip;
            v[i].z = (v[i].z & p.q_keep) ^ p.q_flip;
            v[i].w = (v[i].w & p.q_keep) ^ p.q_flip;
            if constexpr (F8) {
              v[i].x = pack_f16x2(bf16_lo(v[i].x), bf16_hi(v[i].x));
              v[i].y = pack_f16x2(bf16_lo(v[i].y), bf16_hi(v[i].y));
              v[i].z = pack_f16x2(bf16_lo(v[i].z), bf16_hi(v[i].z));
              v[i].w = pack_f16x2(bf16_lo(v[i].w), bf16_hi(v[i].w));
            }
            *reinterpret_cast<uint4*>(dst + (u >> 3) * kPanel + (((u & 7) ^ (row & 7)) << 4)) = v[i];
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      const int step = two ? 1 : 2;
      // A warp without a row of the batch only takes part in the barriers: its rows' weights
      // may be anything, they reach nothing but its rows of O, which nobody reads.
      // (3 sequences on 8k 21.0 -> 18.8 us, 9x4 queries on 32k 74.4 -> 72.7.)
      const bool rows_here = row0 + (two ? w * kPrefixRows : 0) + 32 * (warp & 3) < p.rows;
      float m = -INFINITY, l = 0.f;
      bool alive = true;
      for (int x = t0 + (two ? 0 : w); x < t1; x += step) {
        if (!wait_or_abort(s_full(w), s_phase, p.wait_limit_ns, abort_flag)) {
          alive = false;
          break;
        }
        s_phase ^= 1u;
        tc_fence_after();
        if (!rows_here) {
          float none;
          if (!exchange(0.f, &none)) {
            alive = false;
            break;
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(w));
          continue;
        }
        float s[64];
        tmem_load32(*reinterpret_cast<uint32_t(*)[32]>(&s[0]), s_addr + 64u * half);
        tmem_load32(*reinterpret_cast<uint32_t(*)[32]>(&s[32]), s_addr + 64u * half + 32u);
        tmem_wait_load();
        const int nvalid = p.prefix_tokens - x * kPrefixTokens - 64 * half;
        if (nvalid < 64) {  // the prefix's last tile
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= nvalid) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 60; i += 8)
#pragma unroll
          for (int j = 0; j < 4; ++j) mx[j] = fmaxf(fmaxf(mx[j], s[i + j]), s[i + 4 + j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = fmaxf(mx[j], s[60 + j]);
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])), theirs;
        // Behind the exchange both threads of every row have read their scores,
        // which the weights may now overwrite.
        if (!exchange(top, &theirs)) {
          alive = false;
          break;
        }
        top = fmaxf(top, theirs);
        if (m == -INFINITY) m = top;  // nothing but zero weights so far
        const bool moves = (top - m) * p.scale_log2 > kSlack;
        if (__any_sync(0xffffffffu, moves)) {
          // The products of the group's earlier tiles are done (the scores were
          // issued behind them), so O can be scaled here, half its columns each.
          const float f = moves ? ex2_ftz((m - top) * p.scale_log2) : 1.f;
          if (moves) m = top;
          l *= f;
          if (x >= t0 + step) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[16];
              tmem_load16(o, o_addr + 16u * c);
              tmem_wait_load();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_store16(o_addr + 16u * c, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : kUp - m * p.scale_log2;
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), neg2 = pair(neg, neg);
        uint64_t sum[2] = {0ull, 0ull};
        // The weights enter the product as bf16: half a step, 2^-8 at most, both
        // signs alike; the sum keeps them in fp32.  Where one row tile is all
        // (fine), and the copies set the pace, their remainders follow as a second
        // bf16 part (2^-16 together) in the columns behind.
        auto weights = [&](int e, int i) -> uint32_t {  // two of them, kept in s for their remainders
          float a, b;
          unpair(fma_pair(pair(s[e], s[e + 1]), scale2, neg2), a, b);
          s[e] = ex2_ftz(a);
          s[e + 1] = ex2_ftz(b);
          sum[i & 1] = add_pair(sum[i & 1], pair(s[e], s[e + 1]));
          return F8 ? pack_f16x2(s[e], s[e + 1]) : pack_bf16x2(s[e], s[e + 1]);
        };
        if (!fine) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t hi[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) hi[i] = weights(32 * c + 2 * i, i);
            tmem_store16(s_addr + 32u * half + 16u * c, hi);
          }
        } else {
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int e = 8 * c + 2 * i;
              hi[i] = weights(e, i);
              lo[i] = pack_bf16x2(s[e] - bf16_lo(hi[i]), s[e + 1] - bf16_hi(hi[i]));
            }
            tmem_store4(s_addr + 32u * half + 4u * c, hi);
            tmem_store4(s_addr + 64u + 32u * half + 4u * c, lo);
          }
        }
        {
          float a, b;
          unpair(add_pair(sum[0], sum[1]), a, b);
          l += a + b;
        }
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(w));
      }
      if (alive) alive = wait_or_abort(o_full(w), o_phase, p.wait_limit_ns, abort_flag);
      float theirs = 0.f;
      if (alive) {
        o_phase ^= 1u;
        tc_fence_after();
        alive = exchange(l, &theirs);
      }
      if (!alive) {
        timed_out();
        break;
      }
      const size_t at = ((size_t)(cta + item) * 2 + w) * kPrefixRows + row;
      if (rows_here && half == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(m * p.scale_log2 - kUp, l + theirs);
      if (tid == 0) {
        if (t0 == 0) p.item_ctas[item].x = cta;
        if (t1 == wk.tiles) p.item_ctas[item].y = cta;
      }
      if (rows_here && t0 + (two ? 0 : w) < t1) {  // this group had a tile
        float4* dst = reinterpret_cast<float4*>(p.part_o) + (at - row) * (D / 4) + (D / 8) * half * kPrefixRows + row;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint32_t o[32];
          tmem_load32(o, o_addr + 32u * c);
          tmem_wait_load();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(8 * c + i) * kPrefixRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                         __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
    }
  } else if (warp == kLoadWarp) {
    // ---------------- loads ----------------
    if (lane == 0) {
      prefetch_tensormap(&p.tm_k);
      prefetch_tensormap(&p.tm_v);
    }
    // Stages the copies land in: panels, or the codes of FP8 pools.
    constexpr int kCopyStages = F8 ? NR : NS, kBoxPanels = F8 ? 1 : L::kPanels;
    constexpr uint32_t kCopyBytes = F8 ? L::kRawBytes : L::kTileBytes, kCopyRing = F8 ? L::kRaw : L::kRing;
    auto landed = [&](int i) { return F8 ? raw_full(i) : full(i); };
    auto taken = [&](int i) { return F8 ? raw_empty(i) : empty(i); };
    const int boxes = kPrefixTokens / p.box_rows;
    const int box = lane / kBoxPanels, panel = lane % kBoxPanels;
    const bool mine = box < boxes;
    const uint32_t dst0 = panel * kPanel + box * p.box_rows * (F8 ? (uint32_t)D : 128u);
    Ring ring;
    uint32_t armed = 0, armed_phase = 0;  // stages armed, with the parity of their last phase
    bool alive = true;
    for (int item = first_item; alive && item < wk.items() && wk.item_start(item) < ub; ++item) {
      const int t0 = wk.tile_at(item, ua), t1 = wk.tile_at(item, ub);
      if (t0 >= t1) continue;
      const int head = item / wk.pairs;
      // Token row of this lane's box in tile x, -1 for none (zeros then).
      auto box_row = [&](int x) -> int {
        const int tok = x * kPrefixTokens + box * p.box_rows;
        if (!mine || x >= t1 || tok >= p.prefix_tokens) return -1;
        const int blk = tok / p.block_size, phys = __ldg(p.table + blk);
        if (p.num_physical_blocks > 0 && (phys < 0 || phys >= p.num_physical_blocks)) {
          report(p.error_flag, PA_DEVERR_BLOCK_ID);
          return -1;
        }
        return phys * p.block_size + (tok - blk * p.block_size);
      };
      auto load = [&](const void* tmap, int row, bool withhold) -> bool {
        if (!wait_or_abort(taken(ring.i), ring.phase ^ 1u, p.wait_limit_ns, abort_flag)) {
          timed_out();
          return false;
        }
        if (!withhold) {
          if (lane == 0) mbar_arrive_expect_tx(landed(ring.i), kCopyBytes);
          __syncwarp();
          // A chunk beyond the row's last is outside the tensor: zeros, without a read.
          if (mine)
            tma_load_3d(base + kCopyRing + ring.i * kCopyBytes + dst0, tmap, 0,
                        (row < 0 ? wk.kv_heads : head) * kBoxPanels + panel, row < 0 ? 0 : row, landed(ring.i));
          armed |= 1u << ring.i;
          armed_phase = (armed_phase & ~(1u << ring.i)) | (ring.phase << ring.i);
        }
        ring.next(kCopyStages);
        return true;
      };
      const int ahead = wk.weight(item) == 2 ? 1 : 2;  // K tiles ahead of the V tile
      auto stalls = [&](int x) { return (long long)item * wk.tiles + x == p.stall_tile; };
      int row_v = box_row(t0), row_v1 = box_row(t0 + 1), row_k;
      alive = load(&p.tm_k, row_v, stalls(t0));
      if (alive && ahead == 2 && t0 + 1 < t1) alive = load(&p.tm_k, row_v1, stalls(t0 + 1));
      row_k = ahead == 2 ? box_row(t0 + 2) : row_v1;
      for (int x = t0; alive && x < t1; ++x) {
        const int row_next = box_row(x + ahead + 1);
        alive = load(&p.tm_v, row_v, stalls(x));
        if (alive && x + ahead < t1) alive = load(&p.tm_k, row_k, stalls(x + ahead));
        row_v = row_v1;
        row_v1 = ahead == 2 ? row_k : row_next;
        row_k = row_next;
      }
    }
    named_barrier_sync(1, kPrefixThreads);
    if (*abort_flag != 0) {
      // Copies that were started may still be landing: wait for them (again
      // bounded) before the CTA's shared memory goes.
      for (int i = 0; i < kCopyStages; ++i)
        if ((armed >> i) & 1u) (void)mbar_wait(landed(i), (armed_phase >> i) & 1u, p.wait_limit_ns);
    }
  } else if (warp == kProductWarp) {
    // ---------------- products ----------------
    constexpr uint32_t kScores = product(!F8, 128, 128, false), kValues = product(!F8, 128, D, true);
    Ring ring;
    uint32_t q_phase = 0, p_phase[2] = {0u, 0u};
    bool alive = true;
    const uint64_t q_op = smem_operand(base + L::kQ, kPanel);
    for (int item = first_item; alive && item < wk.items() && wk.item_start(item) < ub; ++item) {
      const int t0 = wk.tile_at(item, ua), t1 = wk.tile_at(item, ub);
      if (t0 >= t1) continue;
      const bool two = wk.weight(item) == 2;
      const int ahead = two ? 1 : 2;
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        if (wait_or_abort(bar, parity, p.wait_limit_ns, abort_flag)) return true;
        timed_out();
        return false;
      };
      // S of group w from the K tile in stage `st`.
      auto scores = [&](int w, int st) {
        if (lane == 0) {
          const uint64_t a = q_op + (two ? (w * L::kTileBytes) >> 4 : 0u);
          const uint64_t b = smem_operand(base + L::kRing + st * L::kTileBytes, kPanel);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = ((k >> 2) * kPanel + (k & 3) * 32u) >> 4;
            mma_ss(tmem + 128u * w, a + off, b + off, kScores, k > 0);
          }
          mma_commit(s_full(w));
        }
        __syncwarp();
      };
      auto release = [&](int st) {
        if (lane == 0) mma_commit(empty(st));
        __syncwarp();
      };
      if (!(alive = wait(q_full, q_phase))) break;
      q_phase ^= 1u;
      tc_fence_after();
      // The first K tiles.
      for (int x = t0; x < t0 + ahead && x < t1; ++x) {
        if (!(alive = wait(full(ring.i), ring.phase))) break;
        tc_fence_after();
        scores(two ? 0 : x - t0, ring.i);
        if (two) scores(1, ring.i);
        release(ring.i);
        ring.next(NS);
      }
      for (int x = t0; alive && x < t1; ++x) {
        const Ring v = ring;
        ring.next(NS);
        const Ring k = ring;
        const bool more = x + ahead < t1;
        if (more) ring.next(NS);
        for (int j = 0; j < (two ? 2 : 1); ++j) {
          const int w = two ? j : (x - t0) & 1;
          if (j == 0 && !(alive = wait(full(v.i), v.phase))) break;
          if (!(alive = wait(p_full(w), p_phase[w]))) break;
          p_phase[w] ^= 1u;
          tc_fence_after();
          if (lane == 0) {
            const uint64_t b = smem_operand(base + L::kRing + v.i * L::kTileBytes, kPanel);
#pragma unroll
            for (int kk = 0; kk < kPrefixTokens / 16; ++kk)
              mma_ts(tmem + 256u + (uint32_t)D * w, tmem + 128u * w + 8u * kk, b + ((kk * 2048u) >> 4), kValues,
                     kk > 0 || x >= t0 + (two ? 1 : 2));
            if (fine) {  // the weights' second part
#pragma unroll
              for (int kk = 0; kk < kPrefixTokens / 16; ++kk)
                mma_ts(tmem + 256u + (uint32_t)D * w, tmem + 128u * w + 64u + 8u * kk, b + ((kk * 2048u) >> 4), kValues,
                       true);
            }
          }
          __syncwarp();
          if (more) {
            if (j == 0 && !(alive = wait(full(k.i), k.phase))) break;
            tc_fence_after();
            scores(w, k.i);
          }
        }
        if (!alive) break;
        release(v.i);
        if (more) release(k.i);
      }
      if (!alive) break;
      if (lane == 0) {
        mma_commit(o_full(0));
        mma_commit(o_full(1));
      }
      __syncwarp();
    }
    // Everything issued is done before tensor memory is freed.
    if (lane == 0) mma_commit(drained);
    __syncwarp();
    (void)mbar_wait_warp(drained, 0, p.wait_limit_ns);
    named_barrier_sync(1, kPrefixThreads);
    tc_fence_after();
    tmem_free(tmem, 512);
    return;
  } else if (F8) {
    // ---------------- codes to f16 ----------------
    // Tiles come in the order of the copies and leave in that of the products,
    // which is the same.  A thread takes 8 codes, a 16-byte unit of a panel row; units
    // of a row lie side by side in a warp, so neither side has bank conflicts.
    constexpr int kThreads = 32 * kWidenWarps, kUnits = D / 8, kSteps = kPrefixTokens * kUnits / kThreads;
    const int t = (warp - kWidenWarp) * 32 + lane, row0 = t / kUnits, unit = t % kUnits;
    Ring ring, raw;
    bool alive = true;
    for (int item = first_item; alive && item < wk.items() && wk.item_start(item) < ub; ++item) {
      const int tiles = 2 * (wk.tile_at(item, ub) - wk.tile_at(item, ua));  // K and V
      for (int x = 0; x < tiles; ++x) {
        alive = wait_or_abort(raw_full(raw.i), raw.phase, p.wait_limit_ns, abort_flag) &&
                wait_or_abort(empty(ring.i), ring.phase ^ 1u, p.wait_limit_ns, abort_flag);
        if (!alive) {
          timed_out();
          break;
        }
        const unsigned char* src = smem + L::kRaw + raw.i * L::kRawBytes + 8 * t;
        unsigned char* dst = smem + L::kRing + ring.i * L::kTileBytes + (unit >> 3) * kPanel + row0 * 128;
        // Loads of a batch go before its stores, which the compiler may not know to be
        // elsewhere: 320 -> 242 us for 256 sequences of 64 heads on 32k (bf16: 256).
        constexpr int kBatch = 8;
        for (int i0 = 0; i0 < kSteps; i0 += kBatch) {
          uint2 codes[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) codes[i] = *reinterpret_cast<const uint2*>(src + 8 * kThreads * (i0 + i));
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = (i0 + i) * (kThreads / kUnits);  // rows from row0
            uint4 v;
            e4m3x4_to_f16x2x2(codes[i].x, v.x, v.y);
            e4m3x4_to_f16x2x2(codes[i].y, v.z, v.w);
            *reinterpret_cast<uint4*>(dst + r * 128 + (((unit & 7) ^ ((row0 + r) & 7)) << 4)) = v;
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full(ring.i));
          mbar_arrive(raw_empty(raw.i));
        }
        ring.next(NS);
        raw.next(NR);
      }
    }
  }
  if (warp < kSoftmaxWarps || warp > kProductWarp) {  // (bf16: the last two warps only fill their warpgroup)
    tc_fence_before();
    named_barrier_sync(1, kPrefixThreads);
  }
}

// ---------------------------------------------------------------------------
// Join: kWarps warps per output row add the row's partials by log-sum-exp: those
// of the prefix, when its sequence shares it, and those of the rest.  The maxima and
// sums of up to 32 partials of either kind are read at once, one per lane; what
// bounds it is the chain of dependent loads, so the lists go side by side, and few
// rows, whose lists are long, get all 8 warps of a CTA.
// ---------------------------------------------------------------------------
struct JoinParams {
  __nv_bfloat16* out;
  const int32_t* context_lens;
  const float* part_ml;
  const float* part_o;
  const float* rest_ml;
  const float* rest_o;
  const int4* cuts;  // the walk's, and its partials
  const float* walk_ml;
  const float* walk_o;
  const int2* item_ctas;
  PrefixWork work;
  int32_t* error_flag;
  int walk_ranges;
  int rows;  // num_seqs * num_queries * num_heads
  int num_queries, num_heads, group, prefix_tokens, max_tokens;
  float v_scale;
};

template <int D, int kWarps>
__global__ void __launch_bounds__(256) pa_prefix_join(const __grid_constant__ JoinParams p) {
  constexpr int kLanes = D / 4;  // lanes that hold four dims (the others repeat them)
  const int lane = threadIdx.x & 31, dims = lane % kLanes, warp = threadIdx.x >> 5, part = warp % kWarps;
  const int row = blockIdx.x * (8 / kWarps) + warp / kWarps;
  if (row >= p.rows) return;  // (all warps of a row alike)
  const int token = row / p.num_heads, h = row - token * p.num_heads;
  const int seq = token / p.num_queries, kv = h / p.group;
  const int r = token * p.group + (h - kv * p.group);  // row of the KV head
  const bool prefix = p.work.tiles > 0;
  const int item = prefix ? kv * p.work.pairs + r / (2 * kPrefixRows) : 0;
  const int in_pair = r % (2 * kPrefixRows);
  const bool two = prefix && p.work.weight(item) == 2;
  griddep_wait();
  griddep_launch_dependents();
  const int4 cut = __ldcg(p.cuts + seq);
  const int c = min(__ldg(p.context_lens + seq), p.max_tokens);
  const int2 ctas = prefix ? __ldcg(p.item_ctas + item) : make_int2(0, -1);
  // Prefix partials: every CTA between the first and the last tile's has one (a
  // range holds two units or more), with a single row tile one per group.
  // (After a timeout of the prefix kernel the table may hold anything: stay inside.)
  const int c0 = max(0, min(ctas.x, p.work.ctas)), c1 = max(-1, min(ctas.y, p.work.ctas - 1));
  const int np = prefix && c >= p.prefix_tokens + p.num_queries - 1 ? max(c1 - c0 + 1, 0) * (two ? 1 : 2) : 0;
  // Partials of the rest: none, the walk's finished row, or one per range.
  const bool whole = cut.w == kCutWhole, holds = cut_holds(cut.x, cut.y, cut.z, cut.w, p.walk_ranges);
  if (!holds && lane == 0) report(p.error_flag, PA_DEVERR_STATE);
  const int nr = !holds || cut.w == kCutEmpty ? 0 : whole ? 1 : cut.y - cut.x + 1;
  const float* ml_r = whole ? p.rest_ml : p.walk_ml;
  const float* o_r = whole ? p.rest_o : p.walk_o;
  const int seq_rows = p.num_queries * p.num_heads, in_seq = row - seq * seq_rows;
  auto rest_at = [&](int k) -> size_t {
    return whole ? (size_t)row : ((size_t)(cut.x + k) * 2 + (k == 0 ? cut.z : 0)) * seq_rows + in_seq;
  };
  auto part_at = [&](int k) -> int { return (c0 + (two ? k : k >> 1) + item) * 2 + (two ? in_pair >> 7 : k & 1); };
  float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  // Partial k of either list belongs to the row's warp k % kWarps; lane j holds the
  // statistics of its j-th.
  auto o_of_part = [&](int k) {
    return __ldcg(reinterpret_cast<const float4*>(p.part_o) +
                  ((size_t)part_at(k) * (D / 4) + dims) * kPrefixRows + (in_pair & 127));
  };
  auto o_of_rest = [&](int k) { return __ldcg(reinterpret_cast<const float4*>(o_r + rest_at(k) * D) + dims); };
  constexpr int kAhead = 8;  // O parts loaded beside the statistics, whatever their weights
  for (int k0 = part; k0 < max(nr, np); k0 += 32 * kWarps) {
    const int k = k0 + lane * kWarps;
    const int here_r = min(32, (nr - k0 + kWarps - 1) / kWarps), here_p = min(32, (np - k0 + kWarps - 1) / kWarps);
    float2 a = make_float2(-INFINITY, 0.f), b = a;
    if (k < nr) a = __ldcg(reinterpret_cast<const float2*>(ml_r) + rest_at(k));
    if (k < np) b = __ldcg(reinterpret_cast<const float2*>(p.part_ml) + (size_t)part_at(k) * kPrefixRows + (in_pair & 127));
    float4 first_r = make_float4(0.f, 0.f, 0.f, 0.f), first_p[kAhead];
    if (here_r > 0) first_r = o_of_rest(k0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < here_p) first_p[i] = o_of_part(k0 + i * kWarps);
    if (a.y == 0.f) a.x = -INFINITY;  // no token seen: no weight
    if (b.y == 0.f) b.x = -INFINITY;
    float top = fmaxf(a.x, b.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float mn = fmaxf(m, top), ref = mn == -INFINITY ? 0.f : mn;
    const float keep = ex2_ftz(m - ref);
    const float wa = ex2_ftz(a.x - ref), wb = ex2_ftz(b.x - ref);
    m = mn;
    float lw = wa * a.y + wb * b.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, o);
    l = l * keep + lw;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] *= keep;
    // A partial without weight may hold anything.
    auto add = [&](float w, const float4& o) {
      if (w != 0.f) {
        acc[0] = fmaf(w, o.x, acc[0]), acc[1] = fmaf(w, o.y, acc[1]);
        acc[2] = fmaf(w, o.z, acc[2]), acc[3] = fmaf(w, o.w, acc[3]);
      }
    };
    if (here_r > 0) add(__shfl_sync(0xffffffffu, wa, 0), first_r);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < here_p) add(__shfl_sync(0xffffffffu, wb, i), first_p[i]);
#pragma unroll 8
    for (int i = 1; i < here_r; ++i) add(__shfl_sync(0xffffffffu, wa, i), o_of_rest(k0 + i * kWarps));
#pragma unroll 8
    for (int i = kAhead; i < here_p; ++i) add(__shfl_sync(0xffffffffu, wb, i), o_of_part(k0 + i * kWarps));
  }
  if constexpr (kWarps > 1) {
    __shared__ float parts[8][6][32];
    float(*mine)[6][32] = parts + (warp - part);  // the row's warps
    mine[part][4][lane] = m;
    mine[part][5][lane] = l;
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[part][i][lane] = acc[i];
    named_barrier_sync(1 + warp / kWarps, 32 * kWarps);
    if (part != 0) return;
#pragma unroll
    for (int w = 1; w < kWarps; ++w) m = fmaxf(m, mine[w][4][lane]);
    const float ref = m == -INFINITY ? 0.f : m;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2_ftz(mine[w][4][lane] - ref);
      l = fmaf(f, mine[w][5][lane], l);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] = fmaf(f, mine[w][i][lane], acc[i]);
    }
  }
  if (lane < kLanes) {
    const float inv = l == 0.f ? 0.f : p.v_scale / l;
    *reinterpret_cast<uint2*>(p.out + (size_t)row * D + 4 * lane) =
        make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Scratch: the rest's (m, l) and O rows, the prefix's partials, then what the
// rest's walk needs.
struct PrefixScratch {
  size_t item_ctas, rest_ml, rest_o, part_ml, part_o, walk, total;
};

PrefixScratch prefix_scratch(int num_seqs, int num_queries, int num_heads, int head_size, int slots,
                             int items, size_t walk_bytes) {
  const size_t rows = (size_t)num_seqs * num_queries * num_heads;
  const size_t part_rows = (size_t)slots * 2 * kPrefixRows;
  PrefixScratch s;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes, 256);
    return at;
  };
  s.item_ctas = take(sizeof(int2) * (size_t)items);
  s.rest_ml = take(rows * 8);
  s.rest_o = take(rows * head_size * 4);
  s.part_ml = take(part_rows * 8);
  s.part_o = take(part_rows * head_size * 4);
  s.walk = take(walk_bytes);
  s.total = o;
  return s;
}

// Items of the list; its slots are at most these and one per SM.
int count_items(int num_seqs, int num_queries, int num_heads, int num_kv_heads) {
  const int64_t rows = (int64_t)num_seqs * num_queries * (num_heads / num_kv_heads);
  const int64_t pairs = (rows + 2 * kPrefixRows - 1) / (2 * kPrefixRows);
  return (int)(pairs * num_kv_heads);
}

// The pools' tensor maps, encoded for every call (about 0.1 us each).
int make_maps(PrefixParams* prm, const void* k, const void* v, uint64_t pool_rows, int num_kv_heads, int head_size,
              bool kv_fp8) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return fail(PA_ERR_CUDA, "pa_decode_prefix: the driver has no cuTensorMapEncodeTiled");
  const cuuint64_t row = (cuuint64_t)num_kv_heads * head_size;
  const cuuint64_t chunk = kv_fp8 ? head_size : 64, elt = kv_fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {chunk, row / chunk, pool_rows}, strides[2] = {chunk * elt, row * elt};
  const cuuint32_t box[3] = {(cuuint32_t)chunk, 1, (cuuint32_t)prm->box_rows}, estride[3] = {1, 1, 1};
  for (int i = 0; i < 2; ++i) {
    const CUresult r = in_context([&] {
      return enc(i ? &prm->tm_v : &prm->tm_k,
                 kv_fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                 const_cast<void*>(i ? v : k), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 kv_fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
    if (r != CUDA_SUCCESS)
      return fail(PA_ERR_CUDA, "pa_decode_prefix: cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  }
  return PA_OK;
}

template <int D, bool F8>
int launch_prefix(const PrefixParams& prm, int device, cudaStream_t stream) {
  static RaisedDevices raised;
  constexpr int kBytes = PrefixLayout<D, F8>::kBytes;
  const int rc = raise_smem_limit(reinterpret_cast<const void*>(pa_prefix_kernel<D, F8>), kBytes, device, &raised);
  if (rc != PA_OK) return rc;
  const cudaError_t e =
      launch_pdl(pa_prefix_kernel<D, F8>, dim3(prm.work.ctas), dim3(kPrefixThreads), kBytes, stream, prm);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "launch pa_prefix_kernel");
}

// Scratch of the walk behind the prefix, whatever the pool's type.
size_t rest_bytes(int num_seqs, int num_queries, int num_heads, int num_kv_heads, int head_size) {
  const size_t bf16 = walk_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, 0, num_queries, 2, false);
  const size_t fp8 = walk_workspace_size(num_seqs, num_heads, num_kv_heads, head_size, 0, num_queries, 1, false);
  return bf16 > fp8 ? bf16 : fp8;
}

}  // namespace
}  // namespace pa

extern "C" size_t pa_decode_prefix_workspace_size(int num_seqs, int num_queries, int num_heads, int num_kv_heads,
                                                  int head_size) {
  using namespace pa;
  const size_t walk = rest_bytes(num_seqs, num_queries, num_heads, num_kv_heads, head_size);
  DeviceInfo dev{};
  if (walk == 0 || current_device_info(&dev) != PA_OK) return 0;
  const int items = count_items(num_seqs, num_queries, num_heads, num_kv_heads);
  return kTicketRoom +
         prefix_scratch(num_seqs, num_queries, num_heads, head_size, dev.sm_count + items, items, walk).total;
}

namespace pa {
namespace {

// What goes before the walk: the prefix kernel, if there is a prefix.
struct PrefixLaunch {
  PrefixParams* prm;
  int head_size;
  bool kv_fp8;
  int device;
  cudaStream_t stream;

  static int run(DecodeExtras* ex, void* context) {
    const PrefixLaunch& l = *static_cast<PrefixLaunch*>(context);
    // The stalled tile of a test: the prefix kernel's tiles come first, then the walk's.
    take_wait_test(&ex->stall_tile, &ex->wait_limit_ns);
    l.prm->stall_tile = -1;
    l.prm->wait_limit_ns = kWaitLimitNs;
    const PrefixWork& w = l.prm->work;
    const long long tiles = w.tiles > 0 ? (long long)w.items() * w.tiles : 0;
    if (ex->stall_tile >= tiles) {
      ex->stall_tile -= tiles;
    } else if (ex->stall_tile >= 0) {
      std::swap(ex->stall_tile, l.prm->stall_tile);
      std::swap(ex->wait_limit_ns, l.prm->wait_limit_ns);
    }
    if (tiles == 0) return PA_OK;
    if (l.kv_fp8)
      return l.head_size == 64 ? launch_prefix<64, true>(*l.prm, l.device, l.stream)
                               : launch_prefix<128, true>(*l.prm, l.device, l.stream);
    return l.head_size == 64 ? launch_prefix<64, false>(*l.prm, l.device, l.stream)
                             : launch_prefix<128, false>(*l.prm, l.device, l.stream);
  }
};

int prefix_impl(void* out, const void* query, const void* k_cache, const void* v_cache, const int32_t* prefix_table,
                const int32_t* block_tables, const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                int num_kv_heads, int head_size, int block_size, int num_prefix_blocks, int max_blocks_per_seq,
                float scale, void* stream, int num_physical_blocks, void* workspace, size_t workspace_bytes,
                int32_t* error_flag, bool kv_fp8, float k_scale, float v_scale) {
  if (num_prefix_blocks < 0 || (num_prefix_blocks > 0 && prefix_table == nullptr))
    return fail(PA_ERR_INVALID_ARG, "pa_decode_prefix: %d prefix blocks without a table", num_prefix_blocks);
  if (num_prefix_blocks > max_blocks_per_seq)
    return fail(PA_ERR_INVALID_ARG, "pa_decode_prefix: prefix of %d blocks in tables of %d", num_prefix_blocks,
                max_blocks_per_seq);
  if (!aligned(prefix_table, 4)) return fail(PA_ERR_INVALID_ARG, "pa_decode_prefix: misaligned prefix_table");
  if (block_size > 0 && block_size % 8 != 0)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode_prefix: block_size %d is not a multiple of 8", block_size);
  int rc = decode_validate(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries,
                           num_heads, num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, PA_BF16,
                           num_physical_blocks);
  if (rc != PA_OK) return rc;
  if (kv_fp8 && (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f))
    return fail(PA_ERR_INVALID_ARG, "pa_decode_fp8_prefix: scales must be finite and positive");
  if (kv_fp8 && num_kv_heads * head_size % 128 != 0)  // as every decode over FP8 pools
    return fail(PA_ERR_UNSUPPORTED, "pa_decode_fp8_prefix: head_size 64 needs an even number of KV heads");
  DeviceInfo dev{};
  rc = current_device_info(&dev);
  if (rc != PA_OK) return rc;
  const size_t walk_bytes = rest_bytes(num_seqs, num_queries, num_heads, num_kv_heads, head_size);
  const int64_t rows = (int64_t)num_seqs * num_queries * (num_heads / num_kv_heads);
  if (rows * num_kv_heads > 1 << 30)
    return fail(PA_ERR_UNSUPPORTED, "pa_decode_prefix: %lld output rows", (long long)(rows * num_kv_heads));
  const int items = count_items(num_seqs, num_queries, num_heads, num_kv_heads);
  const PrefixScratch sc =
      prefix_scratch(num_seqs, num_queries, num_heads, head_size, dev.sm_count + items, items, walk_bytes);
  ScratchHold hold;  // scratch of the library's own, until the launches are queued
  if (workspace == nullptr) {
    rc = hold.of_stream(sc.total, stream, &workspace);
    if (rc != PA_OK) return rc;
  } else {
    if (workspace_bytes < kTicketRoom + sc.total)
      return fail(PA_ERR_WORKSPACE, "pa_decode_prefix: workspace of %zu bytes, %zu needed", workspace_bytes,
                  kTicketRoom + sc.total);
    if (!aligned(workspace, 256))
      return fail(PA_ERR_INVALID_ARG, "pa_decode_prefix: workspace not 256-byte aligned");
    workspace = static_cast<unsigned char*>(workspace) + kTicketRoom;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int prefix_tokens = num_prefix_blocks * block_size;
  const int group = num_heads / num_kv_heads;
  PrefixParams prm{};
  if (num_prefix_blocks > 0) {
    const uint64_t pool_rows =
        num_physical_blocks > 0 ? (uint64_t)num_physical_blocks * block_size
                                : rows_of_pools(k_cache, v_cache, (uint64_t)num_kv_heads * head_size * (kv_fp8 ? 1 : 2));
    if (pool_rows == 0) return PA_ERR_INVALID_ARG;
    if (pool_rows > 1ull << 31)
      return fail(PA_ERR_UNSUPPORTED, "pa_decode_prefix: %llu token rows in the pool (at most 2^31)",
                  (unsigned long long)pool_rows);
    prm.box_rows = block_size & -block_size;
    if (prm.box_rows > kPrefixTokens) prm.box_rows = kPrefixTokens;
    rc = make_maps(&prm, k_cache, v_cache, pool_rows, num_kv_heads, head_size, kv_fp8);
    if (rc != PA_OK) return rc;
    prm.q = static_cast<const __nv_bfloat16*>(query);
    prm.table = prefix_table;
    prm.error_flag = error_flag;
    prm.part_ml = reinterpret_cast<float*>(ws + sc.part_ml);
    prm.part_o = reinterpret_cast<float*>(ws + sc.part_o);
    prm.work = make_prefix_work(rows, num_kv_heads, prefix_tokens, dev.sm_count);
    if (prm.work.ctas == 0)
      return fail(PA_ERR_UNSUPPORTED, "pa_decode_prefix: %lld query rows over %d prefix tokens", (long long)rows,
                  prefix_tokens);
    Plan walk{};
    rc = make_plan(PlanShape{num_heads, num_kv_heads, head_size, num_queries, kv_fp8 ? 1 : 2, 2, block_size}, num_seqs, 0,
                   dev, true, &walk);
    if (rc != PA_OK) return rc;
    prm.item_ctas = reinterpret_cast<int2*>(ws + sc.item_ctas);
    prm.context_lens = context_lens;
    prm.num_seqs = num_seqs;
    prm.num_queries = num_queries;
    prm.max_tokens = max_blocks_per_seq * block_size;
    prm.walk_groups = walk.HG;
    prm.walk_row_bytes = (int)walk.row_bytes;
    prm.sm_count = dev.sm_count;
    prm.rows = (int)rows;
    prm.group = group;
    prm.num_heads = num_heads;
    prm.block_size = block_size;
    prm.prefix_tokens = prefix_tokens;
    prm.num_physical_blocks = num_physical_blocks;
    prm.scale_log2 = scale != 0.f ? (float)(std::fabs((double)scale) * k_scale * 1.4426950408889634) : 1.f;
    prm.q_keep = scale != 0.f ? 0xffffffffu : 0u;
    prm.q_flip = scale < 0.f ? 0x80008000u : 0u;
  }
  DecodeExtras ex{};
  ex.walk = kWalkRest;
  PrefixLaunch first{&prm, head_size, kv_fp8, dev.device, st};
  ex.before = PrefixLaunch::run;
  ex.context = &first;
  ex.prefix_tokens = prefix_tokens;
  ex.rest_ml = reinterpret_cast<float*>(ws + sc.rest_ml);
  ex.rest_o = reinterpret_cast<float*>(ws + sc.rest_o);
  ex.prefix_units = num_prefix_blocks > 0 ? prefix_cost(prm.work) : 0.f;
  rc = decode_impl_q(out, query, k_cache, v_cache, block_tables, context_lens, num_seqs, num_queries, num_heads,
                     num_kv_heads, head_size, block_size, max_blocks_per_seq, scale, stream, PA_BF16,
                     num_physical_blocks, ws + sc.walk, walk_bytes, 0, error_flag, kv_fp8, k_scale, v_scale, nullptr,
                     nullptr, nullptr, &ex);
  if (rc != PA_OK) return rc;
  JoinParams jp{};
  jp.out = static_cast<__nv_bfloat16*>(out);
  jp.context_lens = context_lens;
  jp.part_ml = prm.part_ml;
  jp.part_o = prm.part_o;
  jp.rest_ml = ex.rest_ml;
  jp.rest_o = ex.rest_o;
  jp.cuts = ex.cuts;
  jp.walk_ml = ex.part_ml;
  jp.walk_o = ex.part_o;
  jp.item_ctas = prm.item_ctas;
  jp.work = prm.work;
  jp.error_flag = error_flag;
  jp.walk_ranges = ex.ranges;
  jp.rows = num_seqs * num_queries * num_heads;
  jp.num_queries = num_queries;
  jp.num_heads = num_heads;
  jp.group = group;
  jp.prefix_tokens = prefix_tokens;
  jp.max_tokens = max_blocks_per_seq * block_size;
  jp.v_scale = v_scale;
  // The fewer the rows, the longer their lists and the more warps there are for each.
  // One / two / eight warps a row, whole call: 96 rows (3 sequences on 8k) 32.2 / 24.6 /
  // 21.0 us, 1024 rows 37.2 / 33.3 / 36.7, 2048 rows 38.7 / 39.1 / 48.0, 4096 rows
  // 39.8 / 42.0 / 61.4.
  const int warps = jp.rows <= 4 * dev.sm_count ? 8 : jp.rows <= 16 * dev.sm_count ? 2 : 1;
  const dim3 grid((unsigned)((jp.rows + 8 / warps - 1) / (8 / warps)));
  cudaError_t e;
  if (head_size == 64)
    e = warps == 8   ? launch_pdl(pa_prefix_join<64, 8>, grid, dim3(256), 0, st, jp)
        : warps == 2 ? launch_pdl(pa_prefix_join<64, 2>, grid, dim3(256), 0, st, jp)
                     : launch_pdl(pa_prefix_join<64, 1>, grid, dim3(256), 0, st, jp);
  else
    e = warps == 8   ? launch_pdl(pa_prefix_join<128, 8>, grid, dim3(256), 0, st, jp)
        : warps == 2 ? launch_pdl(pa_prefix_join<128, 2>, grid, dim3(256), 0, st, jp)
                     : launch_pdl(pa_prefix_join<128, 1>, grid, dim3(256), 0, st, jp);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "launch pa_prefix_join");
}

}  // namespace
}  // namespace pa

extern "C" int pa_decode_prefix(void* out, const void* query, const void* k_cache, const void* v_cache,
                                const int32_t* prefix_table, const int32_t* block_tables,
                                const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                                int num_kv_heads, int head_size, int block_size, int num_prefix_blocks,
                                int max_blocks_per_seq, float scale, void* stream, int dtype,
                                int num_physical_blocks, void* workspace, size_t workspace_bytes,
                                int32_t* error_flag) {
  pa::clear_error();
  if (dtype != PA_BF16) return pa::fail(PA_ERR_UNSUPPORTED, "pa_decode_prefix: bf16 only (FP8: pa_decode_fp8_prefix)");
  return pa::prefix_impl(out, query, k_cache, v_cache, prefix_table, block_tables, context_lens, num_seqs,
                         num_queries, num_heads, num_kv_heads, head_size, block_size, num_prefix_blocks,
                         max_blocks_per_seq, scale, stream, num_physical_blocks, workspace, workspace_bytes, error_flag,
                         false, 1.f, 1.f);
}

extern "C" int pa_decode_fp8_prefix(void* out, const void* query, const void* k_cache, const void* v_cache,
                                    const int32_t* prefix_table, const int32_t* block_tables,
                                    const int32_t* context_lens, int num_seqs, int num_queries, int num_heads,
                                    int num_kv_heads, int head_size, int block_size, int num_prefix_blocks,
                                    int max_blocks_per_seq, float scale, float k_scale, float v_scale, void* stream,
                                    int num_physical_blocks, void* workspace, size_t workspace_bytes,
                                    int32_t* error_flag) {
  pa::clear_error();
  return pa::prefix_impl(out, query, k_cache, v_cache, prefix_table, block_tables, context_lens, num_seqs,
                         num_queries, num_heads, num_kv_heads, head_size, block_size, num_prefix_blocks,
                         max_blocks_per_seq, scale, stream, num_physical_blocks, workspace, workspace_bytes, error_flag,
                         true, k_scale, v_scale);
}
