// Attention of chunks of new tokens over the paged cache (pa_prefill,
// pa_prefill_int8, pa_decode_int8).
//
// The (token, group head) rows of a chunk are the rows of two matrix products
// per KV head and tile of 128 tokens, S = Q K^T and O += P V with the running
// statistics of a softmax between them (s in log2 units):
//
//   l_r = sum_t 2^(s_rt - m_r), O_r = sum_t 2^(s_rt - m_r) v_t, out_r = O_r / l_r
//
// for any m_r that no s_rt exceeds: here the maximum over the tiles up to some one, plus 16
// (kSlack), and a later one's where that falls short.
//
// int8 pools: k_t = ks_t * codes, v_t = vs_t * codes.  The codes go through the
// products as they are (every integer up to 256 is a bf16 number), s_rt is
// multiplied by ks_t and the weight by vs_t on its way into the second product.
//
// One persistent CTA per SM, equal shares of the list of (item, tile) units
// (pa_chunk_work.h).  Per CTA:
//   warps 0-3, 4-7  softmax groups 0 and 1: a thread per row, 64 tokens a step; scores
//                   come from tensor memory, weights go back there as bf16
//   warp 8          walks the list, loads queries (TMA) and K and V tiles: TMA boxes of gcd(block_size, 128)
//                   token rows x 64 elements into 128-byte swizzled panels (int8: the
//                   codes into a ring of their own, the scales beside them);
//                   blocks that are no multiple of 8: 16-byte asynchronous copies
//   warp 9          issues the products (tcgen05.mma, one thread)
//   warp 10         bf16: zeroes what lies behind a context's end in its last V tile (zero
//                   weights do not cancel the NaN that may lie there)
//   warps 12-15     int8: widen the codes into the panels
// With two row tiles each group has one and both use every K/V tile; with a
// single row tile the groups take alternate K/V tiles and add their results in
// the end through tensor memory.  A group has two score buffers of 64 tokens: while
// it exponentiates one, the tensor core fills the other, so that neither waits for the
// other's step.  Tensor memory: the buffers (2 x 64 columns a group; the weights overwrite
// the first 32 of one, their second parts, if any, the other 32), O0, O1 (D columns).
//
// What bounds it, and what it measured:
//   long chunks  the tensor core.  4096 tokens on 12,288 others (32 heads on 8, 128 dims):
//                679 us, 1.42 PFLOP/s of the products that the mask leaves.  A tile and its two row
//                tiles need 2,050 clocks of it if S has N = 128, but S in halves of 64 tokens reads
//                its query operand twice as often and takes 1.5 times as long: 2,930 with the
//                commits, which is what the kernel's tiles take.  (S with N = 128 in one buffer a
//                group, a group's softmax under the other's products: not tried.)
//   short items  what an item costs besides its tiles, about 10,000 clocks: first scores, last product,
//                rows out, much of it instruction fetches (0.85 stalls for an instruction per issue,
//                0.53 in long chunks).  7 prompts of 33 to 2,047 tokens: 95 us, 0.68 PFLOP/s; 19
//                single tokens, 3 chunks of 200 to 256 tokens and 2 idle rows on up to 4,096
//                others: 76 us, 2.5 TB/s.
//   few tokens   the chain of a launch: schedule, copies, one tile per CTA, join.  16 on 1k: 19 us.
//   int8         the softmax warps' issue slots, which the widening warps share: a scale into every score
//                and one into every weight.  51% of all slots are used.  4 chunks
//                of 300 to 1,024 tokens on 1k to 7k others and 2 single tokens: 185 us.
#include "pa_launch.cuh"

#include <cmath>
#include <utility>

#include "../../include/pa_int8_cache.h"
#include "pa_chunk.cuh"
#include "pa_decode_impl.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

// Registers per thread at launch: 168 of 384 threads, 128 of 512 (int8); a softmax thread
// holds 64 scores and 32 weights.  256 * 200 + 128 * 104 = 384 * 168, 256 * 176 + 256 * 80 = 512 * 128.
template <bool I8>
struct ChunkWarps {
  static constexpr int kThreads = I8 ? 512 : 384;
  static constexpr int kSoftmaxRegisters = I8 ? 176 : 200, kIssueRegisters = I8 ? 80 : 104;
};
// Place of 16-byte unit u of token row r in a K or V tile.
template <int D>
__device__ __forceinline__ uint32_t unit_at(int r, int u) {
  return (uint32_t)((r >> 3) * (D / 64 * 1024) + (u >> 3) * 1024 + (r & 7) * 128 + (((u & 7) ^ (r & 7)) << 4));
}
constexpr int kSoftmaxWarps = 8, kLoadWarp = 8, kProductWarp = 9, kTailWarp = 10, kWidenWarp = 12, kWidenWarps = 4;
constexpr int kHalf = 64;  // tokens of a softmax step
constexpr uint32_t kPanel = 128 * 128;  // bytes of 128 rows x 64 bf16
// A running maximum is kept until a tile exceeds it by this factor (log2), and weights count
// 2^-16 at the maximum, so that none is above 1 meanwhile: no weight times a value, and no sum of
// them, is larger than by the definition.  bf16 and fp32 hold them as well as 1, down to 2^-110
// of the maximum's.  (With 2^8 a warp of int8 prompts rescaled in every fourth step: 192 us for 185.)
constexpr float kSlack = 16.f;
constexpr int kScaleSlots = 4;  // int8: tiles whose scales are in shared memory
constexpr int kItemSlots = 4;   // items that the loads may be ahead

// An item as the other warps need it; the load warp, which walks the list, puts it into a ring.
struct ChunkItem {
  int row;      // first row of the token buffer
  int tokens;   // of the item; 0: the range has no more items
  int sees;     // tokens that the first of them sees (0 or less: none)
  int head;
  int t0, t1;   // tiles of this CTA
  int ends[2];  // where the steps (halves of tiles) of either group's row tile end
  int flags;
  int ctx, pad[2];
  __device__ __forceinline__ bool two() const { return flags & 1; }    // row tiles
  __device__ __forceinline__ bool whole() const { return flags & 2; }  // no other CTA has a tile
};

template <int D, bool I8>
struct ChunkLayout {
  static constexpr int kPanels = D / 64;
  static constexpr uint32_t kTileBytes = kPanels * kPanel;  // a Q, K or V tile
  // K and V tiles: groups of 8 token rows, a group's panels of 1 KiB side by side, so that
  // the rows of a block come as one copy.  (Q: panels of 128 rows.)
  static constexpr uint32_t kGroup = kPanels * 1024;
  static constexpr int kStages = D == 64 ? 8 : I8 ? 3 : 4;
  static constexpr int kRawStages = I8 ? (D == 64 ? 4 : 2) : 0;  // tiles of codes
  static constexpr uint32_t kRawBytes = kTileBytes / 2;
  static constexpr uint32_t kQ = 1024;  // barriers and items before it
  static constexpr uint32_t kRing = kQ + 2 * kTileBytes;
  static constexpr uint32_t kRaw = kRing + kStages * kTileBytes;
  static constexpr uint32_t kScales = kRaw + kRawStages * kRawBytes;  // [slots][K, V][128] floats
  static constexpr uint32_t kOut = kScales + (I8 ? kScaleSlots * 1024 : 0);  // [softmax warp][32 rows][32 dims] bf16
  static constexpr uint32_t kMl = kOut + kSoftmaxWarps * 2048;               // [group][128] (m, l)
  static constexpr uint32_t kBytes = kMl + 2048;
  static_assert(kBytes <= 227 * 1024, "a CTA's shared memory");
};

__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two codes (the low bytes of the halves of x) as bf16 integers: with the sign bit
// apart, code = (128 + low 7 bits) - (128 or 256), and all three are bf16 numbers of
// one pattern: 0x4300 is 128, and bit 7 of the fraction's carry makes it 256.
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t x) {
  const uint32_t low = (x & 0x007f007fu) | 0x43004300u, sign = (x & 0x00800080u) | 0x43004300u;
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(low), "r"(sign));
  return r;
}

template <int D, bool I8, bool kOdd>
__global__ void __launch_bounds__(ChunkWarps<I8>::kThreads, 1) pa_prefill_kernel(const __grid_constant__ ChunkParams p) {
  using L = ChunkLayout<D, I8>;
  constexpr int NS = L::kStages, NR = L::kRawStages, kChunkThreads = ChunkWarps<I8>::kThreads;
  extern __shared__ __align__(1024) unsigned char smem[];  // swizzled panels start on 1 KiB boundaries
  const uint32_t base = smem_addr(smem);
  if ((base & 1023u) != 0) {  // cannot be: the array asks for it
    if (threadIdx.x == 0) report(p.error_flag, PA_DEVERR_STATE);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t bars = base;
  auto full = [&](int i) { return bars + 8u * i; };
  auto empty = [&](int i) { return bars + 8u * (NS + i); };
  auto tail = [&](int i) { return bars + 8u * (2 * NS + i); };  // a V tile whose end must be zeroed has landed
  auto s_full = [&](int w, int b) { return bars + 8u * (3 * NS + 2 * w + b); };
  auto p_full = [&](int w, int b) { return bars + 8u * (3 * NS + 4 + 2 * w + b); };
  auto o_step = [&](int w) { return bars + 8u * (3 * NS + 8 + w); };  // a step's product has been added
  const uint32_t q_full = bars + 8u * (3 * NS + 10), q_empty = bars + 8u * (3 * NS + 11);
  const uint32_t o_full = bars + 8u * (3 * NS + 12), joined = bars + 8u * (3 * NS + 13);
  const uint32_t drained = bars + 8u * (3 * NS + 14), o_free = bars + 8u * (3 * NS + 15);
  auto sc_full = [&](int i) { return bars + 8u * (3 * NS + 16 + i); };
  auto sc_empty = [&](int i) { return bars + 8u * (3 * NS + 16 + kScaleSlots + i); };
  constexpr int kItemBars = 3 * NS + 16 + 2 * kScaleSlots;
  auto item_full = [&](int i) { return bars + 8u * (kItemBars + i); };
  auto item_empty = [&](int i) { return bars + 8u * (kItemBars + kItemSlots + i); };
  auto raw_full = [&](int i) { return bars + 8u * (kItemBars + 2 * kItemSlots + i); };
  auto raw_empty = [&](int i) { return bars + 8u * (kItemBars + 2 * kItemSlots + NR + i); };
  static_assert(8 * (kItemBars + 2 * kItemSlots + 2 * NR) <= 560, "barriers lie before the flags");
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + 560);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + 564);
  auto timed_out = [&]() {
    if (lane == 0) {
      report(p.error_flag, PA_DEVERR_TIMEOUT);
      *abort_flag = 1;
    }
  };
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), I8 ? kWidenWarps : 1);
      mbar_init(empty(i), 1);
      mbar_init(tail(i), 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(raw_full(i), 1);
      mbar_init(raw_empty(i), kWidenWarps);
    }
    for (int i = 0; i < kScaleSlots; ++i) {
      mbar_init(sc_full(i), 1);
      mbar_init(sc_empty(i), 1);
    }
    for (int i = 0; i < kItemSlots; ++i) {
      mbar_init(item_full(i), 1);
      mbar_init(item_empty(i), kSoftmaxWarps + 1 + (I8 ? kWidenWarps : kOdd ? 0 : 1));
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(o_free, kSoftmaxWarps);
    mbar_init(o_full, 1);
    mbar_init(joined, kSoftmaxWarps);
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full(i >> 1, i & 1), 1);
      mbar_init(p_full(i >> 1, i & 1), kSoftmaxWarps / 2);
    }
    mbar_init(o_step(0), 1);
    mbar_init(o_step(1), 1);
    mbar_init(drained, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  griddep_wait();
  griddep_launch_dependents();

  ChunkItem* ring_items = reinterpret_cast<ChunkItem*>(smem + 576);  // 48 bytes each
  ChunkItems items;
  if (!chunk_begin<kChunkThreads>(p, &items, reinterpret_cast<long long*>(smem + 768))) return;
  // The next item of the ring, and the release of it (by every warp that takes them).
  Ring at_item;
  auto take_item = [&](ChunkItem* it) -> bool {  // false: no more, or a wait ran out
    if (!wait_or_abort(item_full(at_item.i), at_item.phase, p.wait_limit_ns, abort_flag)) {
      timed_out();
      return false;
    }
    const int4* from = reinterpret_cast<const int4*>(ring_items + at_item.i);
    const int4 a = from[0], b = from[1], c = from[2];
    it->row = a.x, it->tokens = a.y, it->sees = a.z, it->head = a.w;
    it->t0 = b.x, it->t1 = b.y, it->ends[0] = b.z, it->ends[1] = b.w;
    it->flags = c.x, it->ctx = c.y;
    return it->tokens > 0;
  };
  auto leave_item = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty(at_item.i));
    at_item.next(kItemSlots);
  };
  if (warp == kProductWarp) tmem_alloc(smem_addr(smem + 564), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kSoftmaxWarps)
    registers_up<ChunkWarps<I8>::kSoftmaxRegisters>();
  else
    registers_down<ChunkWarps<I8>::kIssueRegisters>();

  if (warp < kSoftmaxWarps) {
    // ---------------- softmax ----------------
    const int w = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter of the TMEM lanes
    const uint32_t s_all = tmem + lanes, o_all = s_all + 256u, o_addr = o_all + (uint32_t)D * w;
    uint32_t steps = 0;       // of this group so far: buffer steps & 1, its phase (steps >> 1) & 1
    uint32_t tile_count = 0;  // int8: tiles of the items before (slot and phase of the scales)
    uint32_t o_phase = 0, j_phase = 0;
    bool alive = true;
    const int tok_in = row / p.group;
    ChunkItem it;
    for (; take_item(&it); leave_item()) {
      const bool two = it.two();
      const int row_tile = two ? w : 0;
      const int token = row_tile * p.tile_tokens + tok_in;  // of the item
      const bool real = tok_in < p.tile_tokens && token < it.tokens;
      // Tokens that the row sees.
      const int sees = real ? max(it.sees + token, 0) : 0;
      const int tile_step = two ? 1 : 2, first = 2 * (it.t0 + (two ? 0 : w)), end = w == 0 ? it.ends[0] : it.ends[1];
      // A warp without a row of the batch only takes part in the barriers: its rows' weights
      // may be anything, they reach nothing but its rows of O, which nobody reads.
      const bool rows_here = __any_sync(0xffffffffu, real);
      // Where one row tile is all the copies set the pace, and the weights go in two parts.
      const bool fine = !two;
      float m = -INFINITY, l = 0.f;
      for (int j = first; j < end; j += (j & 1) ? 2 * tile_step - 1 : 1, ++steps) {
        const uint32_t buffer = steps & 1u, s_addr = s_all + 128u * w + 64u * buffer;
        if (!(alive = wait_or_abort(s_full(w, buffer), (steps >> 1) & 1u, p.wait_limit_ns, abort_flag))) break;
        tc_fence_after();
        if (!rows_here) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full(w, buffer));
          continue;
        }
        const float* k_scale = nullptr;
        if constexpr (I8) {
          const uint32_t nth = tile_count + (uint32_t)((j >> 1) - it.t0);
          if (!(alive = wait_or_abort(sc_full(nth % kScaleSlots), (nth / kScaleSlots) & 1u, p.wait_limit_ns, abort_flag)))
            break;
          k_scale = reinterpret_cast<const float*>(smem + L::kScales + (nth % kScaleSlots) * 1024u) + kHalf * (j & 1);
        }
        float s[64];
        tmem_load32(*reinterpret_cast<uint32_t(*)[32]>(&s[0]), s_addr);
        tmem_load32(*reinterpret_cast<uint32_t(*)[32]>(&s[32]), s_addr + 32u);
        tmem_wait_load();
        if (p.sign != 1.f) {  // a negative scale (or zero)
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] *= p.sign;
        }
        if constexpr (I8) {
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(k_scale + i);
            unpair(mul_pair(pair(s[i], s[i + 1]), pair(k4.x, k4.y)), s[i], s[i + 1]);
            unpair(mul_pair(pair(s[i + 2], s[i + 3]), pair(k4.z, k4.w)), s[i + 2], s[i + 3]);
          }
        }
        const int nvalid = sees - j * kHalf;
        const bool masked = nvalid < 64;
        if (masked) {  // tokens behind the row's own
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i >= nvalid) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < 60; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(fmaxf(mx[k], s[i + k]), s[i + 4 + k]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], s[60 + k]);
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        if (m == -INFINITY) m = top;  // nothing but zero weights so far
        const bool moves = (top - m) * p.scale_log2 > kSlack;
        if (__any_sync(0xffffffffu, moves)) {
          const float f = moves ? ex2_ftz((m - top) * p.scale_log2) : 1.f;
          if (moves) m = top;
          l *= f;
          if (j != first) {  // O holds the steps before, once the last of them is added
            if (!(alive = wait_or_abort(o_step(w), (steps - 1) & 1u, p.wait_limit_ns, abort_flag))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D / 16; ++c) {
              uint32_t o[16];
              tmem_load16(o, o_addr + 16u * c);
              tmem_wait_load();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_store16(o_addr + 16u * c, o);
            }
          }
        }
        const float neg = m == -INFINITY ? 0.f : fmaf(-m, p.scale_log2, -kSlack);
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), neg2 = pair(neg, neg);
        uint64_t sum[2] = {0ull, 0ull};
        // The weights enter the product as bf16: half a step, 2^-8 at most, both
        // signs alike; the sum keeps them in fp32.  Where one row tile is all
        // (fine) their remainders follow as a second bf16 part (2^-16 together) in
        // the columns behind.  int8: V's scales go into the weights before the
        // rounding; a scale behind the row's own token, which may be NaN, does not.
        // Half of them at a time, in a loop that stays one: written out, it does not fit the
        // instruction cache beside the other warps' code.
#pragma unroll(I8 ? 1 : 2)
        for (int c = 0; c < 2; ++c) {
          uint32_t hi[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float a, b;
            unpair(fma_pair(pair(s[2 * i], s[2 * i + 1]), scale2, neg2), a, b);
            s[2 * i] = ex2_ftz(a);
            s[2 * i + 1] = ex2_ftz(b);
            sum[i & 1] = add_pair(sum[i & 1], pair(s[2 * i], s[2 * i + 1]));
          }
          if constexpr (I8) {
            const float* v_scale = k_scale + 128 + 32 * c;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 v4 = *reinterpret_cast<const float4*>(v_scale + i);
              unpair(mul_pair(pair(s[i], s[i + 1]), pair(v4.x, v4.y)), s[i], s[i + 1]);
              unpair(mul_pair(pair(s[i + 2], s[i + 3]), pair(v4.z, v4.w)), s[i + 2], s[i + 3]);
            }
            if (masked) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i >= nvalid) s[i] = 0.f;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) hi[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
          tmem_store16(s_addr + 16u * c, hi);
          if (fine) {
#pragma unroll
            for (int i = 0; i < 16; ++i) hi[i] = pack_bf16x2(s[2 * i] - bf16_lo(hi[i]), s[2 * i + 1] - bf16_hi(hi[i]));
            tmem_store16(s_addr + 32u + 16u * c, hi);
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) s[i] = s[32 + i];
        }
        {
          float a, b;
          unpair(add_pair(sum[0], sum[1]), a, b);
          l += a + b;
        }
        tmem_wait_store();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(w, buffer));
      }
      tile_count += (uint32_t)(it.t1 - it.t0);
      if (alive) alive = wait_or_abort(o_full, o_phase, p.wait_limit_ns, abort_flag);
      o_phase ^= 1u;
      tc_fence_after();
      // Whole items end here: a row's thread puts 32 dims at a time where its warp reads
      // them again, and the warp writes its rows out side by side (a thread of a row each
      // would touch 32 lines with every store).  A part of an item leaves its sums for the join.
      const bool whole = it.whole();
      const size_t part = (size_t)2 * blockIdx.x + (it.t0 == 0 ? 1 : 0);
      float* part_o = p.part_o + (part * 2 + row_tile) * (kChunkRows * D) + 4 * row;  // + dims * 128
      float2* part_ml = reinterpret_cast<float2*>(p.part_ml) + part * (2 * kChunkRows) + row_tile * kChunkRows + row;
      float f0 = 1.f, f1 = 0.f;  // factors of this group's O, or of group 0's and group 1's
      int d0 = 0, d1 = D;
      float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
      if (!two) {
        // One row tile: the row's two threads have a part of its tokens each, and take half of
        // the dims each from both groups' O.
        ml[w * kChunkRows + row] = make_float2(m, l);
        __syncwarp();
        if (alive) {
          if (lane == 0) mbar_arrive(joined);
          alive = wait_or_abort(joined, j_phase, p.wait_limit_ns, abort_flag);
          j_phase ^= 1u;
        }
        const float2 a = ml[row], b = ml[kChunkRows + row];
        // A group that saw nothing (l == 0) may have anything in O.
        m = fmaxf(a.y != 0.f ? a.x : -INFINITY, b.y != 0.f ? b.x : -INFINITY);
        f0 = a.y != 0.f ? ex2_ftz((a.x - m) * p.scale_log2) : 0.f;
        f1 = b.y != 0.f ? ex2_ftz((b.x - m) * p.scale_log2) : 0.f;
        l = f0 * a.y + f1 * b.y;
        d0 = (D / 2) * w;
        d1 = d0 + D / 2;
      }
      if (!alive) {
        timed_out();
        break;
      }
      if (rows_here) {
        if (whole || l == 0.f) {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          f0 *= inv;
          f1 *= inv;
        }
        // The rows that this lane writes: 8 i + lane / 4 of the warp's, by the place of their head.
        int place[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = (row & ~31) + 8 * i + (lane >> 2), t = r / p.group, tok = row_tile * p.tile_tokens + t;
          place[i] = t < p.tile_tokens && tok < it.tokens ? (it.row + tok) * p.num_heads + it.head * p.group + (r - t * p.group)
                                                          : -1;
        }
        const uint32_t own = two ? o_addr : o_all;
        unsigned char* staged = smem + L::kOut + warp * 2048;
#pragma unroll 1
        for (int d = d0; d < d1; d += 32) {
          float o[32];
          tmem_load32(*reinterpret_cast<uint32_t(*)[32]>(&o[0]), own + d);
          tmem_wait_load();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = f0 != 0.f ? o[i] * f0 : 0.f;
          if (!two) {
            float more[32];
            tmem_load32(*reinterpret_cast<uint32_t(*)[32]>(&more[0]), own + (uint32_t)D + d);
            tmem_wait_load();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] += f1 != 0.f ? more[i] * f1 : 0.f;
          }
          if (whole) {
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 4; ++u)
              *reinterpret_cast<uint4*>(staged + lane * 64 + ((u ^ ((lane >> 1) & 3)) << 4)) =
                  make_uint4(pack_bf16x2(o[8 * u], o[8 * u + 1]), pack_bf16x2(o[8 * u + 2], o[8 * u + 3]),
                             pack_bf16x2(o[8 * u + 4], o[8 * u + 5]), pack_bf16x2(o[8 * u + 6], o[8 * u + 7]));
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 8 * i + (lane >> 2), u = lane & 3;
              if (place[i] >= 0)
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (size_t)place[i] * D + d + 8 * u) =
                    *reinterpret_cast<const uint4*>(staged + r * 64 + ((u ^ ((r >> 1) & 3)) << 4));
            }
          } else if (real) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<float4*>(part_o + (size_t)(d + 4 * i) * kChunkRows) =
                  make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (!whole && real && (two || w == 0)) *part_ml = make_float2(m * p.scale_log2, l);
      }
      // O, and the places of (m, l), are free for the next item's.
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_free);
    }
  } else if (warp == kLoadWarp) {
    // ---------------- loads ----------------
    if (lane == 0) {
      prefetch_tensormap(&p.tm_q);
      if (!kOdd) {
        prefetch_tensormap(&p.tm_k);
        prefetch_tensormap(&p.tm_v);
      }
    }
    // Stages the copies land in: panels, or the codes of int8 pools.
    constexpr int kCopyStages = I8 ? NR : NS;
    constexpr uint32_t kCopyBytes = I8 ? L::kRawBytes : L::kTileBytes, kCopyRing = I8 ? L::kRaw : L::kRing;
    auto landed = [&](int i) { return I8 ? raw_full(i) : full(i); };
    auto taken = [&](int i) { return I8 ? raw_empty(i) : empty(i); };
    const int boxes = kOdd ? 1 : kChunkTokens / p.box_rows;
    const int box = lane;
    const bool mine = box < boxes;
    const uint32_t dst0 = box * p.box_rows * (I8 ? (uint32_t)D : 2u * D);
    // Block sizes that are powers of two take shifts instead of divisions.
    const int bs_shift = (p.block_size & (p.block_size - 1)) == 0 ? __ffs(p.block_size) - 1 : -1;
    auto block_index = [&](int tok) { return bs_shift >= 0 ? tok >> bs_shift : tok / p.block_size; };
    Ring ring;
    uint32_t armed = 0, armed_phase = 0;       // stages armed, with the parity of their last phase,
    uint32_t tailed = 0, tail_phase = 0;       // and those armed as a tail
    uint32_t scaled = 0, scale_phase = 0;      // slots of scales
    uint32_t queries = 0;                      // items whose queries are asked for
    uint32_t tile_count = 0;
    int late[2] = {-1, -1};  // kOdd: stages whose copies are issued and not yet told of
    bool alive = true;
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      if (wait_or_abort(bar, parity, p.wait_limit_ns, abort_flag)) return true;
      timed_out();
      return false;
    };
    // kOdd: the copies of stage `st` are complete in every lane.
    auto tell = [&](int st) {
      async_proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(landed(st));
    };
    auto tell_all = [&]() {
      copies_wait<0>();
      if (late[0] >= 0) tell(late[0]);
      if (late[1] >= 0) tell(late[1]);
      late[0] = late[1] = -1;
    };
    for (bool more = true; alive && more; more = items.next(p)) {
      if (items.t0 >= items.t1) continue;
      if (!(alive = wait(item_empty(at_item.i), at_item.phase ^ 1u))) break;
      if (lane == 0) {
        const int first = items.pair * 2 * p.tile_tokens;
        int4* to = reinterpret_cast<int4*>(ring_items + at_item.i);
        to[0] = make_int4(items.row.row0 + first, min(items.cs.n - first, 2 * p.tile_tokens), items.cs.old + first + 1,
                          items.head);
        // Steps that the rows up to a token see, one at least.
        auto steps_for = [&](int tokens) {
          const int keys = items.cs.old + min(items.cs.n, tokens);
          return min(2 * items.t1, keys > kHalf ? (keys + kHalf - 1) / kHalf : 1);
        };
        const int end1 = steps_for(first + 2 * p.tile_tokens);
        to[1] = make_int4(items.t0, items.t1, items.two() ? steps_for(first + p.tile_tokens) : end1, end1);
        to[2] = make_int4((items.two() ? 1 : 0) | (items.t0 == 0 && items.t1 == items.tiles ? 2 : 0), items.row.ctx, 0, 0);
        mbar_arrive(item_full(at_item.i));
      }
      __syncwarp();
      at_item.next(kItemSlots);
      const int32_t* table = p.tables + (size_t)items.seq * p.max_blocks;
      const int ctx = items.row.ctx;
      // The block of a token, -1: none (behind the context, or no block of the pool).
      auto entry_of = [&](int tok) -> int { return tok < ctx ? __ldg(table + block_index(tok)) : -1; };
      auto checked = [&](int phys, int tok) -> int {
        if (tok >= ctx || (phys >= 0 && phys < p.num_physical_blocks)) return phys;
        report(p.error_flag, PA_DEVERR_BLOCK_ID);
        return -1;
      };
      auto block_of = [&](int tok) -> int { return checked(entry_of(tok), tok); };
      // The entry of this lane's box in tile x is read well before it is looked at.
      auto box_entry = [&](int x) -> int { return mine && x < items.t1 ? entry_of(x * kChunkTokens + box * p.box_rows) : -1; };
      // Token row of this lane's box in tile x, -1 for none (zeros then).
      auto box_row = [&](int x, int entry) -> int {
        const int tok = x * kChunkTokens + box * p.box_rows;
        if (!mine || x >= items.t1) return -1;
        const int phys = checked(entry, tok);
        return phys < 0 ? -1 : phys * p.block_size + (tok - block_index(tok) * p.block_size);
      };
      // The scales of tile x's tokens.
      auto load_scales = [&](int x, int row, uint32_t nth) -> bool {
        const int slot = nth % kScaleSlots;
        const uint32_t phase = (nth / kScaleSlots) & 1u;
        if (kOdd && __any_sync(0xffffffffu, !mbar_try_wait(sc_empty(slot), phase ^ 1u))) tell_all();
        if (!wait(sc_empty(slot), phase ^ 1u)) return false;
        const uint32_t dst = base + L::kScales + slot * 1024u;
        if constexpr (kOdd) {
          for (int i = 0; i < kChunkTokens; i += 32) {
            const int tok = x * kChunkTokens + i + lane, phys = block_of(tok);
            const size_t at =
                ((size_t)max(phys, 0) * p.kv_heads + items.head) * p.block_size + (tok - block_index(tok) * p.block_size);
            copy_async4(dst + 4u * (i + lane), p.k_scales + at, phys >= 0);
            copy_async4(dst + 512u + 4u * (i + lane), p.v_scales + at, phys >= 0);
          }
          copies_commit();
          tell_all();
          __syncwarp();
          if (lane == 0) mbar_arrive(sc_full(slot));
        } else {
          const bool real = mine && row >= 0;
          const uint32_t bytes = 4u * p.box_rows;
          const unsigned there = __ballot_sync(0xffffffffu, real);
          if (lane == 0) mbar_arrive_expect_tx(sc_full(slot), 2u * bytes * __popc(there));
          __syncwarp();
          if (real) {
            const int phys = block_index(row);
            const size_t at = ((size_t)phys * p.kv_heads + items.head) * p.block_size + (row - phys * p.block_size);
            bulk_copy_g2s(dst + bytes * box, p.k_scales + at, bytes, sc_full(slot));
            bulk_copy_g2s(dst + 512u + bytes * box, p.v_scales + at, bytes, sc_full(slot));
          }
          scaled |= 1u << slot;
          scale_phase = (scale_phase & ~(1u << slot)) | (phase << slot);
        }
        return true;
      };
      auto load = [&](bool v, int x, int row) -> bool {
        const bool withhold = p.stall_tile >= 0 && tile_count + (uint32_t)(x - items.t0) == (uint64_t)p.stall_tile;
        if constexpr (kOdd) {
          // What it waits for may wait for these.
          if (__any_sync(0xffffffffu, !mbar_try_wait(taken(ring.i), ring.phase ^ 1u))) tell_all();
        }
        if (!wait(taken(ring.i), ring.phase ^ 1u)) return false;
        const uint32_t dst = base + kCopyRing + ring.i * kCopyBytes;
        if (withhold) {
        } else if constexpr (kOdd) {
          // 16-byte units of the tile's rows, 32 rows' places at a time.
          constexpr int kUnits = D * (I8 ? 1 : 2) / 16, kRowsAtOnce = 32 / kUnits;
          const unsigned char* pool = static_cast<const unsigned char*>(v ? p.v_cache : p.k_cache);
          const int unit = lane % kUnits;
          for (int r0 = 0; r0 < kChunkTokens; r0 += 32) {
            const int tok = x * kChunkTokens + r0 + lane, phys = block_of(tok);
            const int place = phys < 0 ? -1 : phys * p.block_size + (tok - block_index(tok) * p.block_size);
#pragma unroll 4
            for (int i = 0; i < 32; i += kRowsAtOnce) {
              const int r = i + lane / kUnits, from = __shfl_sync(0xffffffffu, place, r);
              const int rr = r0 + r;
              const uint32_t to = I8 ? (uint32_t)(rr * D + unit * 16) : unit_at<D>(rr, unit);
              copy_async16(dst + to, pool + ((size_t)max(from, 0) * p.kv_heads + items.head) * (16 * kUnits) + unit * 16,
                           from >= 0);
            }
          }
          copies_commit();
          if (late[1] >= 0) {  // the copies before the last two are complete
            copies_wait<2>();
            tell(late[1]);
          }
          late[1] = late[0];
          late[0] = ring.i;
        } else {
          // The rows behind the context's end in its last box are zeroed before V is used.
          const bool ends = !I8 && v && ctx % p.box_rows != 0 && x == (ctx - 1) / kChunkTokens;
          const uint32_t bar = ends ? tail(ring.i) : landed(ring.i);
          if (lane == 0) mbar_arrive_expect_tx(bar, kCopyBytes);
          __syncwarp();
          // A head beyond the last is outside the tensor: zeros, without a read.
          if (mine) {
            const void* map = v ? &p.tm_v : &p.tm_k;
            const int head = row < 0 ? p.kv_heads : items.head, at = row < 0 ? 0 : row;
            if constexpr (I8)
              tma_load_3d(dst + dst0, map, 0, head, at, bar);
            else
              tma_load_5d(dst + dst0, map, 0, 0, 0, at >> 3, head, bar);
          }
          if (ends) {
            tail_phase = (tail_phase & ~(1u << ring.i)) | (((tailed >> ring.i) & 1u ? ~tail_phase & (1u << ring.i) : 0u));
            tailed |= 1u << ring.i;
            armed &= ~(1u << ring.i);
          } else {
            armed |= 1u << ring.i;
            armed_phase = (armed_phase & ~(1u << ring.i)) | (ring.phase << ring.i);
          }
        }
        ring.next(kCopyStages);
        return true;
      };
      const int ahead = items.two() ? 1 : 2;  // K tiles ahead of the V tile
      const int t0 = items.t0, t1 = items.t1;
      // K of tile kx or V of tile vx, whichever the products take next.  Rows of this lane's box in
      // the V tiles vx and vx + 1; the table entry of K's next tile is read a tile before.
      int kx = t0, vx = t0, row_v = -1, row_v1 = -1, entry = kOdd ? -1 : box_entry(t0);
#pragma unroll 1
      while (vx < t1) {
        const bool v = kx >= t1 || kx - vx >= ahead;
        if (v && vx == t0) {
          // The queries, once the item before has all of its scores: (token, group head) rows of a row
          // tile are one box.
          if constexpr (kOdd) tell_all();
          if (queries > 0 && !(alive = wait(q_empty, (queries - 1) & 1u))) break;
          const int copies = (items.two() ? 2 : 1) * L::kPanels;
          if (lane == 0) mbar_arrive_expect_tx(q_full, 128u * p.group * p.tile_tokens * copies);
          __syncwarp();
          if (lane < copies)
            tma_load_3d(base + L::kQ + lane * kPanel, &p.tm_q, 64 * (lane % L::kPanels), items.head * p.group,
                        items.row.row0 + (2 * items.pair + lane / L::kPanels) * p.tile_tokens, q_full);
          ++queries;
        }
        int row = row_v;
        if (!v) {
          if constexpr (!kOdd) {
            row = box_row(kx, entry);
            entry = box_entry(kx + 1);
          }
          if (kx == vx)
            row_v = row;
          else
            row_v1 = row;
          if (I8 && !(alive = load_scales(kx, row, tile_count + (uint32_t)(kx - t0)))) break;
        }
        if (!(alive = load(v, v ? vx : kx, row))) break;
        if (v) {
          ++vx;
          row_v = row_v1;
        } else {
          ++kx;
        }
      }
      tile_count += (uint32_t)(t1 - t0);
    }
    if constexpr (kOdd) tell_all();
    if (alive && wait(item_empty(at_item.i), at_item.phase ^ 1u)) {
      if (lane == 0) {
        ring_items[at_item.i].tokens = 0;  // no more
        mbar_arrive(item_full(at_item.i));
      }
      __syncwarp();
    }
    named_barrier_sync(1, kChunkThreads);
    if (*abort_flag != 0) {
      // Copies that were started may still be landing: wait for them (again
      // bounded) before the CTA's shared memory goes.
      if (queries > 0) (void)mbar_wait(q_full, (queries - 1) & 1u, p.wait_limit_ns);
      for (int i = 0; i < kCopyStages; ++i) {
        if ((armed >> i) & 1u) (void)mbar_wait(landed(i), (armed_phase >> i) & 1u, p.wait_limit_ns);
        if ((tailed >> i) & 1u) (void)mbar_wait(tail(i), (tail_phase >> i) & 1u, p.wait_limit_ns);
      }
      for (int i = 0; i < kScaleSlots; ++i)
        if ((scaled >> i) & 1u) (void)mbar_wait(sc_full(i), (scale_phase >> i) & 1u, p.wait_limit_ns);
    }
  } else if (warp == kProductWarp) {
    // ---------------- products ----------------
    constexpr uint32_t kScores = product(true, 128, kHalf, false), kValues = product(true, 128, D, true);
    Ring ring;
    uint32_t tile_count = 0;
    uint32_t scores_taken[2] = {0u, 0u}, values_taken[2] = {0u, 0u};  // steps of either group
    bool alive = true;
    const uint32_t q_op = smem_operand_low(base + L::kQ, kPanel), elected = elect_one();
    constexpr uint32_t kQHigh = smem_operand_high(1024), kTileHigh = smem_operand_high(L::kGroup);
    constexpr uint32_t kHalfBytes = kHalf / 8 * L::kGroup;
    // Read by every lane, the same in all of them.
    auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = (uint32_t)uniform((int)tmem);
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      if (wait_or_abort(bar, parity, p.wait_limit_ns, abort_flag)) {
        tc_fence_after();
        return true;
      }
      timed_out();
      return false;
    };
    ChunkItem it;
    uint32_t nth = 0;  // item
    for (; alive && take_item(&it); leave_item(), ++nth) {
      const int t0 = uniform(it.t0), t1 = uniform(it.t1), end0 = uniform(it.ends[0]), end1 = uniform(it.ends[1]);
      const bool two = uniform(it.flags) & 1;
      auto release = [&](int st) { mma_commit_warp(empty(st), elected); };
      if (!(alive = wait(q_full, nth & 1u))) break;
      // What follows is written out for both kinds of items, and once more for tiles in whose place
      // nothing ends: one warp issues everything, and its branches take as long as the products.
      auto item_of = [&](auto two_tag) -> bool {
        constexpr bool kTwo = decltype(two_tag)::value;
        constexpr int kStep = kTwo ? 1 : 2;
        auto end = [&](int w) { return w == 0 ? end0 : end1; };
        // The scores of half h of the K tile in stage `st`, for group w.
        auto scores = [&](auto w_tag, int st, int h) {
          constexpr int w = decltype(w_tag)::value;
          const uint32_t buffer = scores_taken[w]++ & 1u;
          const uint32_t a = q_op + (kTwo && w == 1 ? L::kTileBytes >> 4 : 0u);
          const uint32_t b = smem_operand_low(base + L::kRing + st * L::kTileBytes + h * kHalfBytes, 1024u);
          const uint32_t to = tm + 128u * w + 64u * buffer;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss_warp(to, a + (((k >> 2) * kPanel + (k & 3) * 32u) >> 4), kQHigh,
                        b + (((k >> 2) * 1024u + (k & 3) * 32u) >> 4), kTileHigh, kScores, k > 0, elected);
          mma_commit_warp(s_full(w, buffer), elected);
        };
        // Adds the group's weights times half h of the V tile in stage `st`.
        auto values = [&](auto w_tag, int st, int h, bool accumulate) -> bool {
          constexpr int w = decltype(w_tag)::value;
          const uint32_t n = values_taken[w]++, buffer = n & 1u;
          if (!wait(p_full(w, buffer), (n >> 1) & 1u)) return false;
          const uint32_t b = smem_operand_low(base + L::kRing + st * L::kTileBytes + h * kHalfBytes, 1024u);
          const uint32_t o = tm + 256u + (uint32_t)D * w, weights = tm + 128u * w + 64u * buffer;
#pragma unroll
          for (int kk = 0; kk < kHalf / 16; ++kk)
            mma_ts_warp(o, weights + 8u * kk, b + ((kk * 2 * L::kGroup) >> 4), kTileHigh, kValues, kk > 0 || accumulate,
                        elected);
          if constexpr (!kTwo) {  // the weights' second part
#pragma unroll
            for (int kk = 0; kk < kHalf / 16; ++kk)
              mma_ts_warp(o, weights + 32u + 8u * kk, b + ((kk * 2 * L::kGroup) >> 4), kTileHigh, kValues, true, elected);
          }
          mma_commit_warp(o_step(w), elected);
          return true;
        };
        using W0 = std::integral_constant<int, 0>;
        using W1 = std::integral_constant<int, 1>;
        // The first K tile of either group.
#pragma unroll 1
        for (int i = 0; i < kStep && t0 + i < t1; ++i) {
          if (!wait(full(ring.i), ring.phase)) return false;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if ((kTwo || i == 0) && 2 * (t0 + i) + h < end0) scores(W0{}, ring.i, h);
            if ((kTwo || i == 1) && 2 * (t0 + i) + h < end1) scores(W1{}, ring.i, h);
          }
          release(ring.i);
          ring.next(NS);
        }
        // V of tile x and K of the group's next, in steps of half h and group w: with two row tiles
        // the groups in turn, both with both tiles; with one a group's steps and then the other's.
        Ring v, k;
        auto step = [&](auto w_tag, int h, auto inner_tag, int x) -> bool {
          constexpr int w = decltype(w_tag)::value;
          constexpr bool kInner = decltype(inner_tag)::value;  // all of the steps that are asked for exist
          if (!kInner && x >= t1) return true;
          const int next = x + kStep;
          if (h == 0 && (!kTwo || w == 0)) {
            v = ring;
            ring.next(NS);
            k = ring;
            if (kInner || next < t1) ring.next(NS);
            if (!wait(full(v.i), v.phase)) return false;
          }
          if ((kInner || 2 * x + h < end(w)) && !values(w_tag, v.i, h, x > t0 + (kTwo ? 0 : w) || h > 0)) return false;
          if (kInner || (next < t1 && 2 * next + h < end(w))) {
            if (h == 0 && (!kInner || !kTwo || w == 0) && !wait(full(k.i), k.phase)) return false;
            scores(w_tag, k.i, h);
          }
          if (h == 1 && (!kTwo || w == 1)) {
            release(v.i);
            if (kInner || next < t1) {
              // (A tile that no group has a step of is waited for here, before it goes.)
              if (!kInner && !wait(full(k.i), k.phase)) return false;
              release(k.i);
            }
            if (I8) {  // the softmax is done with the tile's scales
              if (lane == 0) mbar_arrive(sc_empty((tile_count + (uint32_t)(x - t0)) % kScaleSlots));
              __syncwarp();
            }
          }
          return true;
        };
        auto steps = [&](auto inner, int x) -> bool {
          if constexpr (kTwo) {
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
              if (!step(W0{}, h, inner, x) || !step(W1{}, h, inner, x)) return false;
          } else {
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
              if (!step(W0{}, h, inner, x)) return false;
#pragma unroll 1
            for (int h = 0; h < 2; ++h)
              if (!step(W1{}, h, inner, x + 1)) return false;
          }
          return true;
        };
        const int inner_end = min(end0, end1);  // steps before it exist for both groups
        // O is the item before's until its rows are out.
        if (nth > 0 && !wait(o_free, (nth - 1) & 1u)) return false;
        for (int x = t0; x < t1; x += kStep) {
          if (x + kStep >= t1) mma_commit_warp(q_empty, elected);  // all scores are asked for
          const int last = x + (kTwo ? 1 : 3);  // tile of the last scores
          if (!(2 * last + 1 < inner_end ? steps(std::true_type{}, x) : steps(std::false_type{}, x))) return false;
        }
        return true;
      };
      alive = two ? item_of(std::true_type{}) : item_of(std::false_type{});
      if (!alive) break;
      tile_count += (uint32_t)(t1 - t0);
      mma_commit_warp(o_full, elected);
    }
    // Everything issued is done before tensor memory is freed.
    mma_commit_warp(drained, elected);
    __syncwarp();
    (void)mbar_wait_warp(drained, 0, p.wait_limit_ns);
    named_barrier_sync(1, kChunkThreads);
    tc_fence_after();
    tmem_free(tmem, 512);
    return;
  } else if (I8 && warp >= kWidenWarp) {
    // ---------------- codes to bf16 ----------------
    // Tiles come in the order of the copies and leave in that of the products,
    // which is the same.  A thread takes 8 codes, a 16-byte unit of a panel row; units
    // of a row lie side by side in a warp, so neither side has bank conflicts.
    constexpr int kThreads = 32 * kWidenWarps, kUnits = D / 8, kSteps = kChunkTokens * kUnits / kThreads;
    const int t = (warp - kWidenWarp) * 32 + lane, row0 = t / kUnits, unit = t % kUnits;
    Ring ring, raw;
    bool alive = true;
    ChunkItem it;
    for (; alive && take_item(&it); leave_item()) {
      const int tiles = 2 * (it.t1 - it.t0);  // K and V
      for (int x = 0; x < tiles; ++x) {
        alive = wait_or_abort(raw_full(raw.i), raw.phase, p.wait_limit_ns, abort_flag) &&
                wait_or_abort(empty(ring.i), ring.phase ^ 1u, p.wait_limit_ns, abort_flag);
        if (!alive) {
          timed_out();
          break;
        }
        const unsigned char* src = smem + L::kRaw + raw.i * L::kRawBytes + 8 * t;
        unsigned char* dst = smem + L::kRing + ring.i * L::kTileBytes;
        // Loads of a batch go before its stores.  (Larger batches do not fit the instruction cache
        // beside the other warps' code: 4 chunks of int8 prompts 212 us, with 8 a batch 227, with 16 268.)
        constexpr int kBatch = 4;
#pragma unroll 1
        for (int i0 = 0; i0 < kSteps; i0 += kBatch) {
          uint2 codes[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) codes[i] = *reinterpret_cast<const uint2*>(src + 8 * kThreads * (i0 + i));
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int r = (i0 + i) * (kThreads / kUnits);  // rows from row0
            uint4 v;
            v.x = codes_to_bf16x2(__byte_perm(codes[i].x, 0u, 0x4140));
            v.y = codes_to_bf16x2(__byte_perm(codes[i].x, 0u, 0x4342));
            v.z = codes_to_bf16x2(__byte_perm(codes[i].y, 0u, 0x4140));
            v.w = codes_to_bf16x2(__byte_perm(codes[i].y, 0u, 0x4342));
            *reinterpret_cast<uint4*>(dst + unit_at<D>(row0 + r, unit)) = v;
          }
        }
        async_proxy_fence();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full(ring.i));
          mbar_arrive(raw_empty(raw.i));
        }
        ring.next(NS);
        raw.next(NR);
      }
    }
  } else if (!I8 && !kOdd && warp == kTailWarp) {
    // ---------------- the end of a context ----------------
    uint32_t at = 0, phases = 0;  // loads of the segments before; parity per stage
    bool alive = true;
    ChunkItem it;
    for (; alive && take_item(&it); leave_item()) {
      at += 2u * (uint32_t)(it.t1 - it.t0);
      const int ctx = it.ctx, x = it.t1 - 1;
      if (ctx % p.box_rows == 0 || x != (ctx - 1) / kChunkTokens) continue;
      const int st = (int)((at - 1) % NS);  // the segment's last load
      if (!(alive = wait_or_abort(tail(st), (phases >> st) & 1u, p.wait_limit_ns, abort_flag))) {
        timed_out();
        break;
      }
      phases ^= 1u << st;
      const int r0 = ctx - x * kChunkTokens, rows = p.box_rows - r0 % p.box_rows;
      for (int i = lane; i < rows * (D / 8); i += 32) {
        const int r = r0 + i / (D / 8), u = i % (D / 8);
        *reinterpret_cast<uint4*>(smem + L::kRing + st * L::kTileBytes + unit_at<D>(r, u)) = make_uint4(0u, 0u, 0u, 0u);
      }
      async_proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(full(st));
    }
  }
  if (warp != kLoadWarp) {
    tc_fence_before();
    named_barrier_sync(1, kChunkThreads);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Tensor maps, encoded for every call (about 0.1 us each): queries (element, head, token) in
// boxes of a row tile's tokens, and the pools.
int make_maps(ChunkParams* prm, uint64_t pool_rows, int head_size, bool int8, bool pools) {
  const EncodeTiledFn enc = encode_tiled_fn();
  if (enc == nullptr) return fail(PA_ERR_CUDA, "pa_prefill: the driver has no cuTensorMapEncodeTiled");
  auto encode = [&](CUtensorMap* map, const void* at, bool bytes, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                    const cuuint32_t* box) -> int {
    const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
    const CUresult r = in_context([&] {
      return enc(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(at),
                 dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                 bytes ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    });
    return r == CUDA_SUCCESS ? PA_OK : fail(PA_ERR_CUDA, "pa_prefill: cuTensorMapEncodeTiled failed (CUresult %d)", (int)r);
  };
  const cuuint64_t d = head_size, row = (cuuint64_t)prm->kv_heads * head_size;
  const cuuint64_t q_dims[3] = {d, (cuuint64_t)prm->num_heads, (cuuint64_t)prm->num_tokens}, q_strides[2] = {2 * d, 2 * d * prm->num_heads};
  const cuuint32_t q_box[3] = {64, (cuuint32_t)prm->group, (cuuint32_t)prm->tile_tokens};
  int rc = encode(&prm->tm_q, prm->q, false, 3, q_dims, q_strides, q_box);
  for (int i = 0; i < 2 && pools && rc == PA_OK; ++i) {
    CUtensorMap* map = i ? &prm->tm_v : &prm->tm_k;
    const void* at = i ? prm->v_cache : prm->k_cache;
    if (int8) {
      const cuuint64_t dims[3] = {d, (cuuint64_t)prm->kv_heads, (cuuint64_t)pool_rows}, strides[2] = {d, row};
      const cuuint32_t box[3] = {(cuuint32_t)d, 1, (cuuint32_t)prm->box_rows};
      rc = encode(map, at, true, 3, dims, strides, box);
    } else {
      // (element of a panel, row of 8, panel, group of 8 rows, head): blocks are multiples of 8 rows here.
      const cuuint64_t dims[5] = {64, 8, d / 64, (cuuint64_t)pool_rows / 8, (cuuint64_t)prm->kv_heads};
      const cuuint64_t strides[4] = {2 * row, 128, 16 * row, 2 * d};
      const cuuint32_t box[5] = {64, 8, (cuuint32_t)(d / 64), (cuuint32_t)prm->box_rows / 8, 1};
      rc = encode(map, at, false, 5, dims, strides, box);
    }
  }
  return rc;
}

template <int D, bool I8, bool kOdd>
int launch_chunks(const ChunkParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  static RaisedDevices raised;
  constexpr int kBytes = ChunkLayout<D, I8>::kBytes;
  const auto kernel = pa_prefill_kernel<D, I8, kOdd>;
  const int rc = raise_smem_limit(reinterpret_cast<const void*>(kernel), kBytes, dev.device, &raised);
  if (rc != PA_OK) return rc;
  cudaError_t e = launch_pdl(kernel, dim3(dev.sm_count), dim3(ChunkWarps<I8>::kThreads), kBytes, stream, prm);
  if (e != cudaSuccess) return cuda_fail(e, "launch pa_prefill_kernel");
  if (dev.sm_count > 1)
    e = launch_pdl(pa_prefill_join<__nv_bfloat16, D>, dim3(dev.sm_count - 1, kJoinBlocks), dim3(256), 0, stream, prm);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "launch pa_prefill_join");
}

}  // namespace

int prefill_validate(const ChunkCall& c) {
  const bool none = c.num_queries == 0 && c.num_tokens == 0;  // whose query and out may be null
  int rc = decode_validate(none ? c.k_cache : c.out, none ? c.k_cache : c.query, c.k_cache, c.v_cache, c.block_tables, c.context_lens, c.num_seqs, 1,
                           c.num_heads, c.num_kv_heads, c.head_size, c.block_size, c.max_blocks_per_seq, c.scale,
                           c.int8 ? PA_BF16 : c.dtype, c.num_physical_blocks);
  if (rc != PA_OK) return rc;
  if (c.num_queries == 0 && (c.seq_starts == nullptr || !aligned(c.seq_starts, 4)))
    return fail(PA_ERR_INVALID_ARG, "pa_prefill: seq_starts is null or misaligned");
  if (c.num_tokens < 0 || c.num_queries < 0)
    return fail(PA_ERR_INVALID_ARG, "pa_prefill: %d tokens, %d queries", c.num_tokens, c.num_queries);
  const long long tokens = c.tokens();
  if (tokens * c.num_heads > 0x7fffffffll)
    return fail(PA_ERR_UNSUPPORTED, "pa_prefill: %lld tokens of %d heads", tokens, c.num_heads);
  if (c.int8) {
    if (c.k_scales == nullptr || c.v_scales == nullptr) return fail(PA_ERR_INVALID_ARG, "pa_prefill_int8: null scales");
    if (!aligned(c.k_scales, 16) || !aligned(c.v_scales, 16))
      return fail(PA_ERR_INVALID_ARG, "pa_prefill_int8: scales must be 16-byte aligned");
    if (c.num_physical_blocks <= 0)
      return fail(PA_ERR_INVALID_ARG, "pa_prefill_int8: num_physical_blocks %d", c.num_physical_blocks);
  }
  return PA_OK;
}

int prefill_impl(const ChunkCall& c) {
  int rc = prefill_validate(c);
  if (rc != PA_OK) return rc;
  const long long tokens = c.tokens();
  if (tokens == 0) return PA_OK;
  DeviceInfo dev{};
  rc = current_device_info(&dev);
  if (rc != PA_OK) return rc;
  const bool f32 = !c.int8 && c.dtype == PA_F32;
  const ChunkScratch sc = chunk_scratch(c.head_size, dev.sm_count);
  ChunkParams prm{};
  prm.k_cache = c.k_cache;
  prm.v_cache = c.v_cache;
  prm.kv_heads = c.num_kv_heads;
  prm.box_rows = c.block_size & -c.block_size;
  if (prm.box_rows > kChunkTokens) prm.box_rows = kChunkTokens;
  const uint64_t pool_rows =
      c.num_physical_blocks > 0
          ? (uint64_t)c.num_physical_blocks * c.block_size
          : rows_of_pools(c.k_cache, c.v_cache, (uint64_t)c.num_kv_heads * c.head_size * (f32 ? 4 : 2));
  if (pool_rows == 0) return PA_ERR_INVALID_ARG;
  if (pool_rows > 1ull << 31)
    return fail(PA_ERR_UNSUPPORTED, "pa_prefill: %llu token rows in the pool (at most 2^31)", (unsigned long long)pool_rows);
  const bool odd = prm.box_rows < 8;
  ScratchHold hold;  // scratch of the library's own, until the launches are queued
  void* workspace = c.workspace;
  if (workspace == nullptr) {
    rc = hold.of_stream(sc.total, c.stream, &workspace);
    if (rc != PA_OK) return rc;
  } else if (c.workspace_bytes < kTicketRoom + sc.total) {
    return fail(PA_ERR_WORKSPACE, "pa_prefill: workspace of %zu bytes, %zu needed", c.workspace_bytes,
                kTicketRoom + sc.total);
  } else if (!aligned(workspace, 256)) {
    return fail(PA_ERR_INVALID_ARG, "pa_prefill: workspace not 256-byte aligned");
  } else {
    workspace = static_cast<unsigned char*>(workspace) + kTicketRoom;
  }
  unsigned char* ws = static_cast<unsigned char*>(workspace);
  prm.q = c.query;
  prm.out = c.out;
  prm.k_scales = c.k_scales;
  prm.v_scales = c.v_scales;
  prm.tables = c.block_tables;
  prm.context_lens = c.context_lens;
  prm.seq_starts = c.num_queries > 0 ? nullptr : c.seq_starts;
  prm.error_flag = c.error_flag;
  prm.cuts = reinterpret_cast<int4*>(ws + sc.cuts);
  prm.part_ml = reinterpret_cast<float*>(ws + sc.part_ml);
  prm.part_o = reinterpret_cast<float*>(ws + sc.part_o);
  prm.num_tokens = (int)tokens;
  prm.num_seqs = c.num_seqs;
  prm.num_queries = c.num_queries;
  prm.num_heads = c.num_heads;
  prm.group = c.num_heads / c.num_kv_heads;
  prm.tile_tokens = (f32 ? kChunkRowsF32 : kChunkRows) / prm.group;
  prm.item_units = f32 ? kItemUnitsF32 : kItemUnits;
  prm.block_size = c.block_size;
  prm.max_blocks = c.max_blocks_per_seq;
  prm.max_tokens = c.max_blocks_per_seq * c.block_size;
  prm.num_physical_blocks = (int)(pool_rows / c.block_size);  // what the rows that the driver knows of hold
  prm.scale_log2 = c.scale != 0.f ? (float)(std::fabs((double)c.scale) * 1.4426950408889634) : 1.f;
  prm.sign = c.scale > 0.f ? 1.f : c.scale < 0.f ? -1.f : 0.f;
  cudaStream_t st = static_cast<cudaStream_t>(c.stream);
  if (f32) {
    prm.scale_log2 = (float)((double)c.scale * 1.4426950408889634);
    return launch_chunks_f32(prm, dev, st, c.head_size);
  }
  rc = make_maps(&prm, pool_rows, c.head_size, c.int8, !odd);
  if (rc != PA_OK) return rc;
  take_wait_test(&prm.stall_tile, &prm.wait_limit_ns);
  if (c.head_size == 64) {
    if (c.int8) return odd ? launch_chunks<64, true, true>(prm, dev, st) : launch_chunks<64, true, false>(prm, dev, st);
    return odd ? launch_chunks<64, false, true>(prm, dev, st) : launch_chunks<64, false, false>(prm, dev, st);
  }
  if (c.int8) return odd ? launch_chunks<128, true, true>(prm, dev, st) : launch_chunks<128, true, false>(prm, dev, st);
  return odd ? launch_chunks<128, false, true>(prm, dev, st) : launch_chunks<128, false, false>(prm, dev, st);
}

}  // namespace pa

extern "C" size_t pa_prefill_workspace_size(int head_size) {
  using namespace pa;
  DeviceInfo dev{};
  if ((head_size != 64 && head_size != 128) || current_device_info(&dev) != PA_OK) return 0;
  return kTicketRoom + chunk_scratch(head_size, dev.sm_count).total;
}

extern "C" int pa_prefill(void* out, const void* query, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens, const int32_t* seq_starts,
                          int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_size, int block_size,
                          int max_blocks_per_seq, float scale, void* stream, int dtype, int num_physical_blocks,
                          void* workspace, size_t workspace_bytes, int32_t* error_flag) {
  pa::clear_error();
  pa::ChunkCall c{};
  c.out = out, c.query = query, c.k_cache = k_cache, c.v_cache = v_cache;
  c.block_tables = block_tables, c.context_lens = context_lens, c.seq_starts = seq_starts;
  c.num_tokens = num_tokens, c.num_seqs = num_seqs, c.num_heads = num_heads, c.num_kv_heads = num_kv_heads;
  c.head_size = head_size, c.block_size = block_size, c.max_blocks_per_seq = max_blocks_per_seq;
  c.scale = scale, c.stream = stream, c.dtype = dtype, c.num_physical_blocks = num_physical_blocks;
  c.workspace = workspace, c.workspace_bytes = workspace_bytes, c.error_flag = error_flag;
  return pa::prefill_impl(c);
}

extern "C" int pa_prefill_int8(void* out, const void* query, const void* k_cache, const void* v_cache,
                               const float* k_scales, const float* v_scales, const int32_t* block_tables,
                               const int32_t* context_lens, const int32_t* seq_starts, int num_tokens, int num_seqs,
                               int num_heads, int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq,
                               float scale, void* stream, int num_physical_blocks, void* workspace,
                               size_t workspace_bytes, int32_t* error_flag) {
  pa::clear_error();
  pa::ChunkCall c{};
  c.int8 = true, c.k_scales = k_scales, c.v_scales = v_scales;
  c.out = out, c.query = query, c.k_cache = k_cache, c.v_cache = v_cache;
  c.block_tables = block_tables, c.context_lens = context_lens, c.seq_starts = seq_starts;
  c.num_tokens = num_tokens, c.num_seqs = num_seqs, c.num_heads = num_heads, c.num_kv_heads = num_kv_heads;
  c.head_size = head_size, c.block_size = block_size, c.max_blocks_per_seq = max_blocks_per_seq;
  c.scale = scale, c.stream = stream, c.dtype = PA_BF16, c.num_physical_blocks = num_physical_blocks;
  c.workspace = workspace, c.workspace_bytes = workspace_bytes, c.error_flag = error_flag;
  return pa::prefill_impl(c);
}
