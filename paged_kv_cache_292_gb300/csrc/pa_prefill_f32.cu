// Chunk attention over fp32 pools (pa_prefill), on the CUDA cores: the list, its
// ranges and the join are those of the bf16 kernel (pa_chunk.cuh), an item is 128
// rows (two row tiles of 64).
//
// A CTA of 256 threads holds the item's queries and 64 tokens' K and V in shared
// memory.  Thread (ty, tx) of 16 x 16 takes rows 8 ty .. 8 ty + 7: their scores for tokens
// tx + 16 j, and their output dims 4 tx + 64 j ...  The statistics of a row are
// shared by its 16 threads, half a warp.  A tile's products are summed by themselves and
// then added, so that a long context's sum is made of few and long steps.
//
// What bounds it is the fp32 pipe and the operands' way to it: K of the next step and V of
// this one come by asynchronous copies behind the arithmetic.  2 x 1000 tokens on 3,000
// others (16 heads on 4, 128 dims) take 1,421 us, 40 TFLOP/s, 54% of what the pipe's 128 lanes
// per SM do; 4 sequences of one token on 8k 266 us, where 4 of an item's 128 rows are real
// (decode of such batches has pa_decode).
#include "pa_chunk.cuh"

namespace pa {
namespace {

constexpr int kF32Threads = 256;
constexpr int kStep = 64;  // tokens in shared memory
constexpr int kItemRows = 2 * kChunkRowsF32;

template <int D>
struct F32Layout {
  static constexpr int kPitch = D + 4;  // floats: 16 rows of one 16-byte unit lie in different banks
  static constexpr uint32_t kQ = 512;   // bytes; the search's words before it
  static constexpr uint32_t kK = kQ + kItemRows * kPitch * 4;
  static constexpr uint32_t kV = kK + kStep * kPitch * 4;
  static constexpr uint32_t kP = kV + kStep * D * 4;
  static constexpr int kPPitch = kStep + 4;
  static constexpr uint32_t kBytes = kP + kItemRows * kPPitch * 4;
};

template <int D>
__global__ void __launch_bounds__(kF32Threads, 1) pa_prefill_f32_kernel(const __grid_constant__ ChunkParams p) {
  using L = F32Layout<D>;
  extern __shared__ __align__(16) unsigned char smem[];
  float* sq = reinterpret_cast<float*>(smem + L::kQ);
  float* sk = reinterpret_cast<float*>(smem + L::kK);
  float* sv = reinterpret_cast<float*>(smem + L::kV);
  float* sp = reinterpret_cast<float*>(smem + L::kP);
  griddep_wait();
  griddep_launch_dependents();
  ChunkItems items;
  if (!chunk_begin<kF32Threads>(p, &items, reinterpret_cast<long long*>(smem))) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  constexpr int kUnits = D / 4;  // 16-byte units of a row
  constexpr int kRowStep = kF32Threads / kUnits, kCopies = kStep / kRowStep;
  // Row 8 ty + i in shared memory: a warp's two rows lie side by side, in different banks.
  auto row_at = [](int ty, int i) { return 16 * i + ty; };
  const float* q = static_cast<const float*>(p.q);
  float* out = static_cast<float*>(p.out);
  // Row i of the item: its token in the chunk (-1: none) and its place in query and out.
  auto token_of = [&](int i, size_t* at) -> int {
    const int tile = i / kChunkRowsF32, r = i % kChunkRowsF32, tok = r / p.group, g = r - tok * p.group;
    const int token = (2 * items.pair + tile) * p.tile_tokens + tok;
    *at = ((size_t)(items.row.row0 + token) * p.num_heads + items.head * p.group + g) * D;
    return r < p.tile_tokens * p.group && token < items.cs.n ? token : -1;
  };
  for (bool more = true; more; more = items.next(p)) {
    if (items.t0 >= items.t1) continue;
    const int32_t* table = p.tables + (size_t)items.seq * p.max_blocks;
    const int ctx = items.row.ctx;
    __syncthreads();  // the item before is done with shared memory
    for (int i = tid; i < kItemRows * kUnits; i += kF32Threads) {
      const int r = i / kUnits, u = i % kUnits;
      size_t at;
      const bool real = token_of(r, &at) >= 0;
      *reinterpret_cast<float4*>(sq + row_at(r >> 3, r & 7) * L::kPitch + 4 * u) =
          real ? __ldg(reinterpret_cast<const float4*>(q + at) + u) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    int sees[8];
    float m[8], l[8], acc[8][D / 16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      size_t at;
      const int token = token_of(8 * ty + i, &at);
      sees[i] = token < 0 ? 0 : max(items.cs.old + token + 1, 0);
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) acc[i][j] = 0.f;
    }
    bool mine = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      size_t at;
      mine = mine || token_of(8 * ty + i, &at) >= 0;
    }
    const bool rows_here = __any_sync(0xffffffffu, mine);
    const int begin = items.t0 * kChunkTokens, end = min(items.t1 * kChunkTokens, ctx);
    // K of a step is copied while the step before multiplies V, V while the scores are
    // made: a buffer each.  A thread copies unit tid % kUnits of rows tid / kUnits + kRowStep i.
    int place[kCopies];  // those rows in the pool (-1: none)
    auto look_up = [&](int t0) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) {
        const int tok = t0 + tid / kUnits + kRowStep * i;
        place[i] = -1;
        if (tok < end) {
          const int blk = tok / p.block_size, phys = __ldg(table + blk);
          if (phys < 0 || phys >= p.num_physical_blocks)
            report(p.error_flag, PA_DEVERR_BLOCK_ID);
          else
            place[i] = phys * p.block_size + (tok - blk * p.block_size);
        }
      }
    };
    auto copy = [&](const void* pool, float* to, int pitch) {
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        copy_async16(smem_addr(to + (tid / kUnits + kRowStep * i) * pitch + 4 * (tid % kUnits)),
                     static_cast<const float4*>(pool) + ((size_t)max(place[i], 0) * p.kv_heads + items.head) * kUnits + tid % kUnits,
                     place[i] >= 0);
    };
    if (begin < end) {
      look_up(begin);
      copy(p.k_cache, sk, L::kPitch);
      copies_commit();
      copy(p.v_cache, sv, D);
    }
    copies_commit();
    for (int t0 = begin; t0 < end; t0 += kStep) {
      const bool more_steps = t0 + kStep < end;
      if (more_steps) look_up(t0 + kStep);
      copies_wait<1>();
      __syncthreads();  // K is there (and the queries)
      float keep[8];
      if (rows_here) {  // (else the warp's 16 rows are none of the chunk's)
        float s[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 2
        for (int u = 0; u < kUnits; ++u) {
          float4 a[8], b[4];
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = *reinterpret_cast<const float4*>(sq + row_at(ty, i) * L::kPitch + 4 * u);
#pragma unroll
          for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * L::kPitch + 4 * u);
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[i][j] = fmaf(a[i].x, b[j].x, s[i][j]);
              s[i][j] = fmaf(a[i].y, b[j].y, s[i][j]);
              s[i][j] = fmaf(a[i].z, b[j].z, s[i][j]);
              s[i][j] = fmaf(a[i].w, b[j].w, s[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float top = -INFINITY;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[i][j] = t0 + tx + 16 * j < sees[i] ? s[i][j] * p.scale_log2 : -INFINITY;
            top = fmaxf(top, s[i][j]);
          }
#pragma unroll
          for (int o = 1; o < 16; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float mn = fmaxf(m[i], top), ref = mn == -INFINITY ? 0.f : mn;
          keep[i] = ex2_ftz(m[i] - ref);
          m[i] = mn;
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float w = ex2_ftz(s[i][j] - ref);
            sum += w;
            sp[row_at(ty, i) * L::kPPitch + tx + 16 * j] = w;
          }
          l[i] = fmaf(l[i], keep[i], sum);
        }
      }
      __syncthreads();  // K is read (and a row's weights are there, which its own half warp reads)
      if (more_steps) copy(p.k_cache, sk, L::kPitch);
      copies_commit();
      copies_wait<1>();
      __syncthreads();  // V is there
      if (rows_here) {
        float part[8][D / 16];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < D / 16; ++j) part[i][j] = 0.f;
#pragma unroll 2
        for (int t = 0; t < kStep; t += 4) {
          float4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = *reinterpret_cast<const float4*>(sp + row_at(ty, i) * L::kPPitch + t);
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
              const float4 v = *reinterpret_cast<const float4*>(sv + (t + e) * D + 64 * j + 4 * tx);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float f = e == 0 ? w[i].x : e == 1 ? w[i].y : e == 2 ? w[i].z : w[i].w;
                part[i][4 * j] = fmaf(f, v.x, part[i][4 * j]);
                part[i][4 * j + 1] = fmaf(f, v.y, part[i][4 * j + 1]);
                part[i][4 * j + 2] = fmaf(f, v.z, part[i][4 * j + 2]);
                part[i][4 * j + 3] = fmaf(f, v.w, part[i][4 * j + 3]);
              }
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < D / 16; ++j) acc[i][j] = fmaf(acc[i][j], keep[i], part[i][j]);
      }
      __syncthreads();  // V is read
      if (more_steps) copy(p.v_cache, sv, D);
      copies_commit();
    }
    copies_wait<0>();
    const bool whole = items.t0 == 0 && items.t1 == items.tiles;
    const size_t part = (size_t)2 * blockIdx.x + (items.t0 == 0 ? 1 : 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], o);
      const int r = 8 * ty + i, tile = r / kChunkRowsF32, in_tile = r % kChunkRowsF32;
      size_t at;
      if (token_of(r, &at) < 0) continue;  // (the whole half warp: one row)
      const float inv = !whole ? 1.f : l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const int d = 64 * j + 4 * tx;
        const float4 v = make_float4(acc[i][4 * j] * inv, acc[i][4 * j + 1] * inv, acc[i][4 * j + 2] * inv, acc[i][4 * j + 3] * inv);
        if (whole)
          *reinterpret_cast<float4*>(out + at + d) = v;
        else
          *reinterpret_cast<float4*>(p.part_o + (part * 2 + tile) * (kChunkRows * D) + (size_t)d * kChunkRows + 4 * in_tile) = v;
      }
      if (!whole && tx == 0)
        reinterpret_cast<float2*>(p.part_ml)[part * (2 * kChunkRows) + tile * kChunkRows + in_tile] = make_float2(m[i], l[i]);
    }
  }
}

template <int D>
int launch(const ChunkParams& prm, const DeviceInfo& dev, cudaStream_t stream) {
  static RaisedDevices raised;
  const auto kernel = pa_prefill_f32_kernel<D>;
  const int rc = raise_smem_limit(reinterpret_cast<const void*>(kernel), F32Layout<D>::kBytes, dev.device, &raised);
  if (rc != PA_OK) return rc;
  cudaError_t e = launch_pdl(kernel, dim3(dev.sm_count), dim3(kF32Threads), F32Layout<D>::kBytes, stream, prm);
  if (e != cudaSuccess) return cuda_fail(e, "launch pa_prefill_f32_kernel");
  if (dev.sm_count > 1)
    e = launch_pdl(pa_prefill_join<float, D>, dim3(dev.sm_count - 1, kJoinBlocks), dim3(256), 0, stream, prm);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, "launch pa_prefill_join");
}

}  // namespace

int launch_chunks_f32(const ChunkParams& prm, const DeviceInfo& dev, cudaStream_t stream, int head_size) {
  return head_size == 64 ? launch<64>(prm, dev, stream) : launch<128>(prm, dev, stream);
}

}  // namespace pa
