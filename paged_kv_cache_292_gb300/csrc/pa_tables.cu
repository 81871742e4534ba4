// Block tables, context lengths and slot maps of one step, built on the GPU
// from the requests' lengths (pa_tables_step).
//
// With base_s the tokens sequence s holds before the step's (its context, or
// the shared prefix for a sequence that starts), n_s its new tokens and bs the
// block size, the step is three running sums over the sequences in order:
//   back_s = blocks a released sequence returns,
//   need_s = ceil((base_s + n_s) / bs) - ceil(base_s / bs) blocks taken,
//   grow_s = n_s slots,
// after which every output entry is a function of its own index: the k-th
// returned block goes to free_blocks[count + k], the k-th taken one comes from
// position top - 1 - k (top = count + sum of back), and slot i belongs to the
// sequence whose interval of grow holds i.
//
// What bounds it is latency: a step reads and writes a few bytes per sequence
// and 8 bytes per slot.  Measured on the device: 3.5 us for 64 sequences with a
// token each (an empty kernel takes 2 to 3), 6.6 for 517 with prompt chunks, 13.5 for
// 4096 with 0.5 M slots (4.7 MB, 0.7 us of HBM time; 10 us of it are the sums over 4096
// sequences, which every CTA redoes because waiting for another's costs as much).  So it is one launch: every CTA redoes the three sums
// over all sequences in shared memory (no CTA waits for another) and then
// takes its share of each output.  A taken block that was returned in the same
// step is read from the table row that returned it, so no CTA reads what
// another one writes.
#include <cuda_runtime.h>

#include "../../include/pa_tables.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

// Few sequences and slots take CTAs of few warps, which start and synchronise
// quickly, many as many threads as an SM holds.  Device time with 256 / 1024 threads:
//   64 sequences, a slot each             3.5 / 5.4 us
//   1024 sequences, a slot each           5.3 / 6.8
//   517 sequences, 25 k slots             6.6 / 8.2
//   256 sequences, 100 k slots            6.0 / 5.9
//   512 sequences, 250 k slots           10.2 / 7.2
//   4096 sequences, a slot each          18.2 / 9.8
//   4096 sequences, 0.5 M slots          29.7 / 13.8
constexpr int kSmallThreads = 256, kLargeThreads = 1024;
constexpr int kTablesMaxSeqs = 12288;  // four int32 per sequence in shared memory

struct TablesParams {
  int32_t* block_tables;
  int32_t* context_lens_out;
  int32_t* seq_starts;
  int64_t* slot_mapping;
  int32_t* free_blocks;
  int32_t* free_count_out;
  const int32_t* context_lens;
  const int32_t* new_lens;
  const int32_t* free_count;
  const int32_t* prefix_table;
  int32_t* error_flag;
  int num_seqs, num_prefix_blocks, max_blocks, block_size, num_physical_blocks, max_tokens;
};

// Sums of v[0..2] over the threads before this one and over all (THREADS / 32 <= 32 warps).
template <int THREADS>
__device__ __forceinline__ void block_sums(long long (&v)[3], long long (&total)[3], long long (&scratch)[3][32],
                                           int lane, int warp) {
  long long incl[3];
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    incl[q] = v[q];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, incl[q], o);
      if (lane >= o) incl[q] += n;
    }
    if (lane == 31) scratch[q][warp] = incl[q];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    const long long mine = lane < THREADS / 32 ? scratch[q][lane] : 0;
    long long sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long n = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += n;
    }
    v[q] = __shfl_sync(0xffffffffu, sum - mine, warp) + incl[q] - v[q];
    total[q] = __shfl_sync(0xffffffffu, sum, 31);
  }
}

// First index s with ends[s] > x (ends is non-decreasing and its last entry is > x).
__device__ __forceinline__ int owner_of(const int* ends, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS) pa_tables_kernel(const TablesParams p) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ long long scratch[3][32], reduce[2][32];
  const int S = p.num_seqs, bs = p.block_size, np = p.num_prefix_blocks;
  int* grow_end = reinterpret_cast<int*>(smem);
  int* need_end = grow_end + S;
  int* back_end = need_end + S;
  int* base_of = back_end + S;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0;
  // Blocks that hold t tokens, and the block of token t (t < 2^30 + 4096).
  const int shift = (bs & (bs - 1)) == 0 ? __ffs(bs) - 1 : -1;
  auto block_of = [&](int t) { return shift >= 0 ? t >> shift : t / bs; };
  auto blocks_for = [&](int t) { return block_of(t + bs - 1); };
  griddep_wait();

  // Per sequence: what it returns, takes and gets, were the pool without end.
  const long long width_tokens = (long long)p.max_blocks * bs;
  int bad = 0;
#pragma unroll 4
  for (int s = tid; s < S; s += THREADS) {
    const int c = __ldg(p.context_lens + s);
    int n = __ldg(p.new_lens + s);
    const long long first_own = (long long)np * bs;
    // A length the table cannot hold, or one that ends inside the prefix.
    if (c < 0 || c > width_tokens || (c > 0 && c < first_own) || n < PA_TABLES_RELEASE) {
      bad |= PA_DEVERR_CONTEXT_LEN;
      n = 0;
    }
    int back = 0, need = 0, base = c;
    if (n == PA_TABLES_RELEASE) {
      back = c > 0 ? blocks_for(c) - np : 0;
      n = 0;
    } else if (n > 0) {
      if (c == 0) base = (int)first_own;
      const long long end = (long long)base + n;
      if (end > width_tokens) {
        bad |= PA_DEVERR_CONTEXT_LEN;
        n = 0;
      } else {
        need = blocks_for((int)end) - blocks_for(base);
      }
    }
    grow_end[s] = n;
    need_end[s] = need;
    back_end[s] = back;
    base_of[s] = base;
  }
  __syncthreads();

  // Running sums: thread t owns the sequences [t * per, (t + 1) * per).
  const int per = (S + THREADS - 1) / THREADS;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  long long grow = 0, need = 0, back = 0;
  for (int s = s0; s < s1; ++s) {
    grow += grow_end[s];
    need += need_end[s];
    back += back_end[s];
  }
  long long sums[3] = {grow, need, back}, total[3];
  block_sums<THREADS>(sums, total, scratch, lane, warp);
  grow = sums[0], need = sums[1], back = sums[2];
  const long long total_back = total[2];
  const int NB = p.num_physical_blocks;
  int count = __ldg(p.free_count);
  if (count < 0 || count > NB) {
    bad |= PA_DEVERR_BLOCK_ID;
    count = count < 0 ? 0 : NB;
  }
  if (count + total_back > NB) bad |= PA_DEVERR_BLOCK_ID;  // more returned than the pool has
  const int top = (int)(count + total_back < NB ? count + total_back : NB);
  // A sequence is served when the sums up to and including it fit; the sums
  // only rise, so the sequences served come before the ones that are not.
  long long served_grow = 0, served_need = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = grow_end[s];
    grow += n;
    need += need_end[s];
    back += back_end[s];
    const bool served = need <= top && grow <= p.max_tokens;
    if (served) {
      served_grow = grow;
      served_need = need;
    } else if (n > 0) {
      bad |= grow > p.max_tokens ? PA_DEVERR_SLOT : PA_DEVERR_NO_BLOCKS;
    }
    grow_end[s] = served ? (int)grow : -1;
    need_end[s] = served ? (int)need : -1;
    back_end[s] = (int)(back < NB ? back : NB);
  }
  // The sums at the last sequence served: the largest over the threads.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    served_grow = max(served_grow, __shfl_xor_sync(0xffffffffu, served_grow, o));
    served_need = max(served_need, __shfl_xor_sync(0xffffffffu, served_need, o));
  }
  if (lane == 0) {
    reduce[0][warp] = served_grow;
    reduce[1][warp] = served_need;
  }
  __syncthreads();
  long long total_grow = lane < THREADS / 32 ? reduce[0][lane] : 0, total_need = lane < THREADS / 32 ? reduce[1][lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total_grow = max(total_grow, __shfl_xor_sync(0xffffffffu, total_grow, o));
    total_need = max(total_need, __shfl_xor_sync(0xffffffffu, total_need, o));
  }
  for (int s = s0; s < s1; ++s) {
    if (grow_end[s] < 0) {
      grow_end[s] = (int)total_grow;
      need_end[s] = (int)total_need;
    }
  }
  __syncthreads();
  griddep_launch_dependents();
  if (first_cta && bad) report(p.error_flag, bad);

  const int gtid = blockIdx.x * THREADS + tid, gthreads = gridDim.x * THREADS;
  const int n_back = (int)(total_back < NB - count ? total_back : NB - count);
  // The block at position i of the free list once the returned ones are on it.
  auto free_block = [&](int i) -> int {
    if (i < count) return __ldg(p.free_blocks + i);
    const int k = i - count, s = owner_of(back_end, S, k);
    return p.block_tables[(size_t)s * p.max_blocks + np + k - (s ? back_end[s - 1] : 0)];
  };

  // Lengths, starts and the prefix's entries of sequences that start.
  for (int sb = gtid - lane; sb < S; sb += gthreads) {
    const int s = sb + lane;
    bool begins = false;
    if (s < S) {
      const int start = s ? grow_end[s - 1] : 0, n = grow_end[s] - start;
      const int c = __ldg(p.context_lens + s);
      begins = n > 0 && c == 0 && np > 0;
      const bool valid = c >= 0 && c <= width_tokens && (c == 0 || c >= (long long)np * bs);
      const bool gone = valid && __ldg(p.new_lens + s) == PA_TABLES_RELEASE;
      p.context_lens_out[s] = n > 0 ? base_of[s] + n : (gone ? 0 : c);
      p.seq_starts[s] = start;
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, begins); todo; todo &= todo - 1) {
      int32_t* row = p.block_tables + (size_t)(sb + __ffs(todo) - 1) * p.max_blocks;
      for (int j = lane; j < np; j += 32) row[j] = __ldg(p.prefix_table + j);
    }
  }
  if (gtid == 0) {
    p.seq_starts[S] = (int)total_grow;
    *p.free_count_out = top - (int)total_need;
  }
  // One list of work for all threads, each entry a chain of searches and loads of
  // its own: the slots, the taken blocks into the tables, the returned ones onto
  // the free list.  (Four slots a thread, which mostly share their block: 4096
  // sequences with 0.5 M slots 16.3 us, one a thread 13.8.)
  const long long slots = p.max_tokens, takes = slots + total_need, all = takes + n_back;
  for (long long entry = gtid; entry < all; entry += gthreads) {
    if (entry >= takes) {
      const int k = static_cast<int>(entry - takes), s = owner_of(back_end, S, k);
      p.free_blocks[count + k] = p.block_tables[(size_t)s * p.max_blocks + np + k - (s ? back_end[s - 1] : 0)];
      continue;
    }
    if (entry >= slots) {
      const int k = static_cast<int>(entry - slots), s = owner_of(need_end, S, k);
      const int j = blocks_for(base_of[s]) + k - (s ? need_end[s - 1] : 0);
      p.block_tables[(size_t)s * p.max_blocks + j] = free_block(top - 1 - k);
      continue;
    }
    const int i = static_cast<int>(entry);
    long long slot = -1;
    if (i < total_grow) {
      const int s = owner_of(grow_end, S, i), base = base_of[s];
      const int pos = base + i - (s ? grow_end[s - 1] : 0), j = block_of(pos), held = blocks_for(base);
      const int b = j < held ? p.block_tables[(size_t)s * p.max_blocks + j]
                             : free_block(top - 1 - ((s ? need_end[s - 1] : 0) + j - held));
      slot = (long long)b * bs + (pos - j * bs);
    }
    p.slot_mapping[i] = slot;
  }
}

template <int THREADS>
int launch_tables(const TablesParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  static RaisedDevices raised;
  const int rc = raise_smem_limit(reinterpret_cast<const void*>(pa_tables_kernel<THREADS>), 16 * kTablesMaxSeqs,
                                  dev.device, &raised);
  if (rc != PA_OK) return rc;
  const long long work = (long long)prm.max_tokens + prm.num_seqs;
  const long long want = (work + THREADS - 1) / THREADS;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(want < dev.sm_count ? want : dev.sm_count));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = 16 * (size_t)prm.num_seqs;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pa_tables_kernel<THREADS>, prm);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "launch pa_tables_kernel");
}

bool overlaps(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

}  // namespace
}  // namespace pa

extern "C" int pa_tables_step(int32_t* block_tables, int32_t* context_lens_out, int32_t* seq_starts,
                              int64_t* slot_mapping, int32_t* free_blocks, int32_t* free_count_out,
                              const int32_t* context_lens, const int32_t* new_lens, const int32_t* free_count,
                              const int32_t* prefix_table, int num_prefix_blocks, int num_seqs,
                              int max_blocks_per_seq, int block_size, int num_physical_blocks, int max_tokens,
                              void* stream, int32_t* error_flag) {
  using namespace pa;
  clear_error();
  if (!block_tables || !context_lens_out || !seq_starts || !free_blocks || !free_count_out || !context_lens ||
      !new_lens || !free_count || (max_tokens > 0 && !slot_mapping) || (num_prefix_blocks > 0 && !prefix_table))
    return fail(PA_ERR_INVALID_ARG, "pa_tables_step: null tensor pointer");
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 || block_size <= 0 || num_physical_blocks <= 0 || max_tokens < 0 ||
      num_prefix_blocks < 0)
    return fail(PA_ERR_INVALID_ARG, "pa_tables_step: sizes must be positive");
  if (num_seqs > kTablesMaxSeqs)
    return fail(PA_ERR_UNSUPPORTED, "pa_tables_step: %d sequences > %d", num_seqs, kTablesMaxSeqs);
  if (block_size > 4096) return fail(PA_ERR_UNSUPPORTED, "pa_tables_step: block_size %d > 4096", block_size);
  if ((long long)max_blocks_per_seq * block_size > (1ll << 30))
    return fail(PA_ERR_INVALID_ARG, "pa_tables_step: max context %lld too large",
                (long long)max_blocks_per_seq * block_size);
  if (num_prefix_blocks > max_blocks_per_seq)
    return fail(PA_ERR_INVALID_ARG, "pa_tables_step: prefix of %d blocks in tables of %d", num_prefix_blocks,
                max_blocks_per_seq);
  if (max_tokens > (1 << 30)) return fail(PA_ERR_INVALID_ARG, "pa_tables_step: max_tokens %d too large", max_tokens);
  if (!aligned(block_tables, 4) || !aligned(context_lens_out, 4) || !aligned(seq_starts, 4) ||
      !aligned(slot_mapping, 8) || !aligned(free_blocks, 4) || !aligned(free_count_out, 4) ||
      !aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(free_count, 4) || !aligned(prefix_table, 4))
    return fail(PA_ERR_INVALID_ARG, "pa_tables_step: misaligned tensor pointer");
  // Every CTA reads the whole input: what one writes must not be what another
  // has still to read, nor what another one writes.
  const size_t S = (size_t)num_seqs;
  const struct { const void* p; size_t n; } out[] = {
      {block_tables, 4 * S * max_blocks_per_seq}, {context_lens_out, 4 * S}, {seq_starts, 4 * (S + 1)},
      {slot_mapping, 8 * (size_t)max_tokens}, {free_blocks, 4 * (size_t)num_physical_blocks}, {free_count_out, 4}},
      in[] = {{context_lens, 4 * S}, {new_lens, 4 * S}, {free_count, 4},
              {prefix_table, 4 * (size_t)num_prefix_blocks}};
  for (size_t i = 0; i < sizeof(out) / sizeof(out[0]); ++i) {
    for (const auto& b : in)
      if (overlaps(out[i].p, out[i].n, b.p, b.n))
        return fail(PA_ERR_INVALID_ARG, "pa_tables_step: an output overlaps an input");
    for (size_t j = i + 1; j < sizeof(out) / sizeof(out[0]); ++j)
      if (overlaps(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(PA_ERR_INVALID_ARG, "pa_tables_step: two outputs overlap");
  }
  DeviceInfo dev{};
  int rc = current_device_info(&dev);
  if (rc != PA_OK) return rc;
  TablesParams prm{block_tables, context_lens_out, seq_starts, slot_mapping, free_blocks, free_count_out,
                   context_lens, new_lens, free_count, prefix_table, error_flag,
                   num_seqs, num_prefix_blocks, max_blocks_per_seq, block_size, num_physical_blocks, max_tokens};
  const size_t smem = 16 * S;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool small = num_seqs <= 1024 && max_tokens <= 2 * dev.sm_count * kSmallThreads;
  return small ? launch_tables<kSmallThreads>(prm, dev, st) : launch_tables<kLargeThreads>(prm, dev, st);
}
