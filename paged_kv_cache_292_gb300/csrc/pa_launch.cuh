// Launching the decode kernel, shared by the translation units that
// instantiate it (one per kind of walk, compiled in parallel).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>

#include "pa_decode_kernel.cuh"
#include "pa_internal.h"
#include "pa_plan.h"

namespace pa {

// Launch with programmatic stream serialisation: the kernel may become
// resident while its predecessor on the stream finishes; it calls
// griddepcontrol.wait before touching anything that predecessor produces.
template <typename Kernel, typename Params>
cudaError_t launch_pdl(Kernel kern, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       const Params& prm) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, prm);
}

template <typename T, int D, int GMAX, int QMODE = 0, bool KV8 = false, int WALK = kWalkAll>
int launch_typed(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream) {
  // Devices whose shared-memory limit is already raised for this kernel
  // (setting it again is harmless, so concurrent first calls may both set it).
  constexpr int kTrackedDevices = 64;
  static std::atomic<bool> configured[kTrackedDevices];
  auto kern = pa_decode_kernel<T, D, GMAX, QMODE, KV8, WALK>;
  if (dev < 0 || dev >= kTrackedDevices || !configured[dev].load(std::memory_order_acquire)) {
    DeviceInfo info{};
    int rc = current_device_info(&info);
    if (rc != PA_OK) return rc;
    const int fixed = WALK == kWalkMod && sizeof(T) == 4 ? kFp32Buffers : 0;  // its static shared memory
    cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, info.max_smem_optin - fixed);
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(decode smem)");
    if (dev >= 0 && dev < kTrackedDevices) configured[dev].store(true, std::memory_order_release);
  }
  cudaError_t e =
      launch_pdl(kern, dim3(pl.R * pl.HG), dim3(32 * (pl.Hg * pl.split + pl.producers)), pl.smem, stream, prm);
  if (e != cudaSuccess) return cuda_fail(e, "launch pa_decode_kernel");
  return PA_OK;
}

// The driver's encoder of tensor maps (nullptr if it has none).
using EncodeTiledFn = PFN_cuTensorMapEncodeTiled_v12000;
EncodeTiledFn encode_tiled_fn();

// `call()`, a call into the driver; where no context is current, as in a host thread
// that has made no CUDA call yet, once more with the device's own.
template <typename Call>
CUresult in_context(Call call) {
  const CUresult r = call();
  int device = 0;
  if (r != CUDA_ERROR_INVALID_CONTEXT || cudaGetDevice(&device) != cudaSuccess || cudaSetDevice(device) != cudaSuccess)
    return r;
  return call();
}

// Token rows for the tensor maps of two pools whose size the caller has not given:
// those the pools' allocations hold behind the pools' addresses, at most 2^31.  0 with an
// error recorded if the driver does not know the memory.
uint64_t rows_of_pools(const void* k, const void* v, uint64_t row_bytes);

// The kernel variants of the other translation units.
int launch_mod(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool f32,
               bool kv_fp8);
int launch_rest(const DecodeParams& prm, const Plan& pl, int dev, cudaStream_t stream, int head_size, bool kv_fp8);

}  // namespace pa
