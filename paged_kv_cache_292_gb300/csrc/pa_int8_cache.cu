// The int8 cache: new rows quantised as they are written (pa_write_cache_int8), and
// tokens read back into plain rows (pa_read_cache_int8).
//
// A row is one token's K or V of one KV head.  Its scale is max |x| / 127 and its
// codes are x / scale rounded to the nearest integer, ties to even.  Whether a
// quotient lies above or below a tie is asked of x - (k + 1/2) scale in one fma,
// whose sign is that of the exact difference, so a code never depends on how a
// quotient was rounded.
//
// A thread has 8 elements, D / 8 threads a row; the K rows of a token come first, then
// its V rows, and a warp takes them in steps, four of them with their loads side by side.
//
// What bounds both kernels is memory.  64 contexts of 512 to 4,096 tokens (8 heads of 128) read to bf16:
// 136 us, 6.7 TB/s read and written together.  4 prompts of 1,000 to 4,099 fp32 rows there and back, 178 MB
// that L2 partly holds: 41 us.  64 tokens there and back: 7.6 us of the GPU's time, two launches.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/pa_int8_cache.h"
#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kCacheThreads = 256;
constexpr int kCacheSteps = 4;  // rows of a thread

template <typename T>
__device__ __forceinline__ void load8(float (&x)[8], const T* src) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(src)), b = __ldg(reinterpret_cast<const float4*>(src) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(src));
    x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
    x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
  }
}

// x / scale to the nearest integer, ties to even, for |x| <= 128 scale.
__device__ __forceinline__ int nearest_code(float x, float scale) {
  if (scale < 0x1p-100f) {  // the difference below must not fall between the smallest numbers
    x *= 0x1p100f;
    scale *= 0x1p100f;
  }
  const float low = floorf(__fdiv_rn(x, scale));
  const float above = fmaf(-(low + 0.5f), scale, x);  // its sign is exact
  const int k = (int)low;
  const int code = above > 0.f ? k + 1 : above < 0.f ? k : k + (k & 1);
  return max(-127, min(127, code));
}

struct WriteParams {
  const void* src[2];
  int8_t* pool[2];
  float* scales[2];
  const int64_t* slots;
  long long num_slots;
  int num_tokens, kv_heads, block_size;
  int32_t* error_flag;
};

template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads) pa_write_int8_kernel(const __grid_constant__ WriteParams p) {
  constexpr int kRowThreads = D / 8, kRowsPerStep = 32 / kRowThreads;
  const int lane = threadIdx.x & 31, unit = lane % kRowThreads;
  const int token = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (token >= p.num_tokens) return;
  const long long slot = __ldg(reinterpret_cast<const long long*>(p.slots) + token);
  if (slot < 0) return;  // padding
  if (slot >= p.num_slots) {
    if (lane == 0 && blockIdx.y == 0) report(p.error_flag, PA_DEVERR_SLOT);
    return;
  }
  const long long block = slot < (1ll << 32) ? (uint32_t)slot / (uint32_t)p.block_size : slot / p.block_size;
  const int in_block = (int)(slot - block * p.block_size);
  const int first = blockIdx.y * (kCacheSteps * kRowsPerStep) + lane / kRowThreads;
  float x[kCacheSteps][8];
#pragma unroll
  for (int i = 0; i < kCacheSteps; ++i) {
    const int r = first + i * kRowsPerStep, v = r >= p.kv_heads, head = r - (v ? p.kv_heads : 0);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
    if (r < 2 * p.kv_heads)
      load8(x[i], static_cast<const T*>(p.src[v]) + ((size_t)token * p.kv_heads + head) * D + 8 * unit);
  }
#pragma unroll
  for (int i = 0; i < kCacheSteps; ++i) {
    const int r = first + i * kRowsPerStep, v = r >= p.kv_heads, head = r - (v ? p.kv_heads : 0);
    // The largest magnitude by its bits, among which infinities and NaN come last.
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[i][e]) & 0x7fffffffu);
#pragma unroll
    for (int o = 1; o < kRowThreads; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool finite = top < 0x7f800000u;
    const float scale = finite ? __fdiv_rn(__uint_as_float(top), 127.f) : __uint_as_float(0x7fc00000u);
    uint2 codes = make_uint2(0u, 0u);
    if (finite && scale > 0.f) {
      // x / scale + 1.5 * 2^23 has the rounded quotient in its low bits.  It is off the
      // nearest integer only next to a tie, where the exact question is asked.
      constexpr float kMagic = 12582912.f;
      const float inv = __frcp_rn(scale);
      uint32_t t[8];
      float far = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = fmaf(x[i][e], inv, kMagic);
        t[e] = __float_as_uint(y);
        far = fmaxf(far, fabsf(fmaf(-(y - kMagic), scale, x[i][e])));
      }
      // (Tiny scales, whose reciprocal or differences are no normal numbers, go the long way.)
      if (!(far < 0.4999f * scale) || scale < 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = (uint32_t)nearest_code(x[i][e], scale);
      }
      codes.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
      codes.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
    }
    if (r < 2 * p.kv_heads) {
      *reinterpret_cast<uint2*>(p.pool[v] + ((size_t)slot * p.kv_heads + head) * D + 8 * unit) = codes;
      if (unit == 0) p.scales[v][((size_t)block * p.kv_heads + head) * p.block_size + in_block] = scale;
    }
  }
}

struct ReadParams {
  void* dst[2];
  const int8_t* pool[2];
  const float* scales[2];
  const int32_t* tables;
  const int32_t* first_tokens;
  const int32_t* seq_starts;
  int num_tokens, num_seqs, kv_heads, block_size, max_blocks, num_physical_blocks;
  int32_t* error_flag;
};

// The number of entries at[0 .. n - 1] (not decreasing) that are <= t, found by a whole warp
// in steps of 32 probes.
__device__ __forceinline__ int count_up_to(const int32_t* at, int n, int t, int lane) {
  int lo = 0, hi = n;  // entries before lo are, those from hi on are not
  while (lo < hi) {
    const int width = (hi - lo + 31) / 32, i = lo + (lane + 1) * width - 1;
    const unsigned below = __ballot_sync(0xffffffffu, i < hi && __ldg(at + i) <= t);
    const int k = __popc(below);
    hi = min(hi, lo + (k + 1) * width - 1);
    lo = min(hi, lo + k * width);
    if (width == 1) break;
  }
  return lo;
}

template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads) pa_read_int8_kernel(const __grid_constant__ ReadParams p) {
  constexpr int kRowThreads = D / 8, kRowsPerStep = 32 / kRowThreads;
  const int lane = threadIdx.x & 31, unit = lane % kRowThreads;
  const int token = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  griddep_wait();
  griddep_launch_dependents();
  if (token >= p.num_tokens) return;
  // The sequence whose rows hold the token: the last that begins at or before it.
  const int s = count_up_to(p.seq_starts, p.num_seqs + 1, token, lane) - 1;
  if (s < 0 || s >= p.num_seqs) return;
  const int from = __ldg(p.seq_starts + s);
  const long long pos = (long long)token - from + (p.first_tokens != nullptr ? __ldg(p.first_tokens + s) : 0);
  const bool report_it = lane == 0 && blockIdx.y == 0;
  // (Among starts that decrease the search may end at a sequence that does not hold the token.)
  if (token < from || token >= __ldg(p.seq_starts + s + 1) || pos < 0 || pos >= (long long)p.max_blocks * p.block_size) {
    if (report_it) report(p.error_flag, PA_DEVERR_CONTEXT_LEN);
    return;
  }
  const int blk = (int)pos / p.block_size, in_block = (int)pos - blk * p.block_size;
  const int phys = __ldg(p.tables + (size_t)s * p.max_blocks + blk);
  if (phys < 0 || phys >= p.num_physical_blocks) {
    if (report_it) report(p.error_flag, PA_DEVERR_BLOCK_ID);
    return;
  }
  const size_t slot = (size_t)phys * p.block_size + in_block;
  const int first = blockIdx.y * (kCacheSteps * kRowsPerStep) + lane / kRowThreads;
  uint2 codes[kCacheSteps];
  float scale[kCacheSteps];
#pragma unroll
  for (int i = 0; i < kCacheSteps; ++i) {
    const int r = first + i * kRowsPerStep, v = r >= p.kv_heads, head = r - (v ? p.kv_heads : 0);
    if (r >= 2 * p.kv_heads) break;
    codes[i] = __ldg(reinterpret_cast<const uint2*>(p.pool[v] + (slot * p.kv_heads + head) * D) + unit);
    scale[i] = __ldg(p.scales[v] + ((size_t)phys * p.kv_heads + head) * p.block_size + in_block);
  }
#pragma unroll
  for (int i = 0; i < kCacheSteps; ++i) {
    const int r = first + i * kRowsPerStep, v = r >= p.kv_heads, head = r - (v ? p.kv_heads : 0);
    if (r >= 2 * p.kv_heads) break;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = (float)(int8_t)((e < 4 ? codes[i].x : codes[i].y) >> (8 * (e & 3))) * scale[i];
    T* dst = static_cast<T*>(p.dst[v]) + ((size_t)token * p.kv_heads + head) * D + 8 * unit;
    if constexpr (sizeof(T) == 4) {
      reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                  pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
  }
}

template <typename Kernel, typename Params>
int launch_rows(Kernel kernel, int num_tokens, int kv_heads, int head_size, const Params& prm, void* stream,
                const char* what) {
  const int per_token = kCacheSteps * (32 / (head_size / 8));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((num_tokens - 1) / (kCacheThreads / 32) + 1),
                     (unsigned)((2 * kv_heads + per_token - 1) / per_token));
  cfg.blockDim = dim3(kCacheThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, prm);
  return e == cudaSuccess ? PA_OK : cuda_fail(e, what);
}

// What both calls ask of their sizes and pools.
int check_sizes(const char* name, const void* k_cache, const void* v_cache, const void* k_scales, const void* v_scales,
                const void* k_rows, const void* v_rows, int num_tokens, int kv_heads, int head_size, int block_size,
                int num_physical_blocks, int dtype) {
  if (!k_cache || !v_cache || !k_scales || !v_scales || (num_tokens > 0 && (!k_rows || !v_rows)))
    return fail(PA_ERR_INVALID_ARG, "%s: null tensor pointer", name);
  if (num_tokens < 0 || kv_heads <= 0 || head_size <= 0 || block_size <= 0 || num_physical_blocks <= 0)
    return fail(PA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (dtype != PA_F32 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "%s: dtype %d", name, dtype);
  if (head_size != 64 && head_size != 128)
    return fail(PA_ERR_UNSUPPORTED, "%s: head_size %d (built: 64, 128)", name, head_size);
  if (block_size > 4096) return fail(PA_ERR_UNSUPPORTED, "%s: block_size %d > 4096", name, block_size);
  if (kv_heads > 65536) return fail(PA_ERR_UNSUPPORTED, "%s: %d KV heads", name, kv_heads);
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scales, 4) || !aligned(v_scales, 4))
    return fail(PA_ERR_INVALID_ARG, "%s: rows and pools must be 16-byte aligned, scales 4-byte", name);
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" int pa_write_cache_int8(const void* k_new, const void* v_new, const int64_t* slot_mapping, void* k_cache,
                                   void* v_cache, float* k_scales, float* v_scales, int num_tokens, int num_kv_heads,
                                   int head_size, int block_size, int num_physical_blocks, void* stream, int src_dtype,
                                   int32_t* error_flag) {
  using namespace pa;
  clear_error();
  const char* name = "pa_write_cache_int8";
  const int rc = check_sizes(name, k_cache, v_cache, k_scales, v_scales, k_new, v_new, num_tokens, num_kv_heads,
                             head_size, block_size, num_physical_blocks, src_dtype);
  if (rc != PA_OK) return rc;
  if (num_tokens > 0 && (slot_mapping == nullptr || !aligned(slot_mapping, 8)))
    return fail(PA_ERR_INVALID_ARG, "%s: slot_mapping is null or misaligned", name);
  if (num_tokens == 0) return PA_OK;
  WriteParams prm{};
  prm.src[0] = k_new, prm.src[1] = v_new;
  prm.pool[0] = static_cast<int8_t*>(k_cache), prm.pool[1] = static_cast<int8_t*>(v_cache);
  prm.scales[0] = k_scales, prm.scales[1] = v_scales;
  prm.slots = slot_mapping;
  prm.num_slots = (long long)num_physical_blocks * block_size;
  prm.num_tokens = num_tokens;
  prm.kv_heads = num_kv_heads;
  prm.block_size = block_size;
  prm.error_flag = error_flag;
  const auto kernel = src_dtype == PA_F32
                          ? (head_size == 64 ? pa_write_int8_kernel<float, 64> : pa_write_int8_kernel<float, 128>)
                          : (head_size == 64 ? pa_write_int8_kernel<__nv_bfloat16, 64> : pa_write_int8_kernel<__nv_bfloat16, 128>);
  return launch_rows(kernel, num_tokens, num_kv_heads, head_size, prm, stream, "launch pa_write_int8_kernel");
}

extern "C" int pa_read_cache_int8(void* k_out, void* v_out, const void* k_cache, const void* v_cache,
                                  const float* k_scales, const float* v_scales, const int32_t* block_tables,
                                  const int32_t* first_tokens, const int32_t* seq_starts, int num_tokens, int num_seqs,
                                  int num_kv_heads, int head_size, int block_size, int max_blocks_per_seq,
                                  int num_physical_blocks, void* stream, int dst_dtype, int32_t* error_flag) {
  using namespace pa;
  clear_error();
  const char* name = "pa_read_cache_int8";
  const int rc = check_sizes(name, k_cache, v_cache, k_scales, v_scales, k_out, v_out, num_tokens, num_kv_heads,
                             head_size, block_size, num_physical_blocks, dst_dtype);
  if (rc != PA_OK) return rc;
  if (block_tables == nullptr || seq_starts == nullptr || !aligned(block_tables, 4) || !aligned(seq_starts, 4) ||
      !aligned(first_tokens, 4))
    return fail(PA_ERR_INVALID_ARG, "%s: tables or seq_starts are null or misaligned", name);
  if (num_seqs <= 0 || max_blocks_per_seq <= 0 || (long long)max_blocks_per_seq * block_size > (1ll << 30))
    return fail(PA_ERR_INVALID_ARG, "%s: %d sequences of %d blocks", name, num_seqs, max_blocks_per_seq);
  if (num_tokens == 0) return PA_OK;
  ReadParams prm{};
  prm.dst[0] = k_out, prm.dst[1] = v_out;
  prm.pool[0] = static_cast<const int8_t*>(k_cache), prm.pool[1] = static_cast<const int8_t*>(v_cache);
  prm.scales[0] = k_scales, prm.scales[1] = v_scales;
  prm.tables = block_tables;
  prm.first_tokens = first_tokens;
  prm.seq_starts = seq_starts;
  prm.num_tokens = num_tokens;
  prm.num_seqs = num_seqs;
  prm.kv_heads = num_kv_heads;
  prm.block_size = block_size;
  prm.max_blocks = max_blocks_per_seq;
  prm.num_physical_blocks = num_physical_blocks;
  prm.error_flag = error_flag;
  const auto kernel = dst_dtype == PA_F32
                          ? (head_size == 64 ? pa_read_int8_kernel<float, 64> : pa_read_int8_kernel<float, 128>)
                          : (head_size == 64 ? pa_read_int8_kernel<__nv_bfloat16, 64> : pa_read_int8_kernel<__nv_bfloat16, 128>);
  return launch_rows(kernel, num_tokens, num_kv_heads, head_size, prm, stream, "launch pa_read_int8_kernel");
}
