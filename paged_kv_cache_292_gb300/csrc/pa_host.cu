// Host-side plumbing: per-thread error messages, cached device properties and
// the library-owned decode scratch.
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>

#include "../../include/pagedattn.h"
#include "pa_internal.h"

namespace pa {

namespace {
thread_local char g_message[512] = {0};
// pa_test_stall_copy: consumed by the next decode launch on this thread.
thread_local long long g_stall_tile = -1;
thread_local unsigned int g_stall_limit_us = 0;

constexpr int kMaxDevices = 64;
std::mutex g_mutex;          // g_info
std::mutex g_scratch_mutex;  // what follows, held by a ScratchHold
DeviceInfo g_info[kMaxDevices];
bool g_info_valid[kMaxDevices] = {false};
void* g_ws_ptr[kMaxDevices] = {nullptr};
size_t g_ws_bytes[kMaxDevices] = {0};
void* g_cnt_ptr[kMaxDevices] = {nullptr};
size_t g_cnt_bytes[kMaxDevices] = {0};
bool g_ws_in_graph[kMaxDevices] = {false}, g_cnt_in_graph[kMaxDevices] = {false};
// ScratchHold::of_stream: a buffer for each of the streams that called last.
struct KeptScratch {
  unsigned long long stream;  // its id, which no other stream of the process ever gets
  unsigned long long used;    // 0: free
  void* ptr;
  size_t bytes;
  void* tickets;  // of decode calls, zero between them
  size_t ticket_bytes;
};
constexpr int kKeptStreams = 8;
KeptScratch g_kept[kMaxDevices][kKeptStreams];
unsigned long long g_kept_calls = 0;
}  // namespace

int fail(int code, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_message, sizeof(g_message), fmt, ap);
  va_end(ap);
  return code;
}

int cuda_fail(cudaError_t err, const char* what) {
  return fail(PA_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(err), cudaGetErrorName(err));
}

void clear_error() { g_message[0] = '\0'; }

int current_device_info(DeviceInfo* info) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(PA_ERR_UNSUPPORTED, "device index %d too large", dev);
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!g_info_valid[dev]) {
    DeviceInfo d{};
    d.device = dev;
    e = cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(sm count)");
    e = cudaDeviceGetAttribute(&d.max_smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
    if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceGetAttribute(smem optin)");
    int major = 0, minor = 0;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (major * 10 + minor != 103)
      return fail(PA_ERR_UNSUPPORTED, "device %d is sm_%d%d; this library is built for sm_103a only",
                  dev, major, minor);
    g_info[dev] = d;
    g_info_valid[dev] = true;
  }
  *info = g_info[dev];
  return PA_OK;
}

int ScratchHold::plain(size_t bytes, size_t counter_bytes, void* stream, void** ptr, int32_t** counters) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  e = cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &status);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  lock_ = std::unique_lock<std::mutex>(g_scratch_mutex);
  if (g_ws_bytes[dev] < bytes) {
    if (g_ws_ptr[dev] != nullptr) {
      e = g_ws_in_graph[dev] ? cudaSuccess : cudaFree(g_ws_ptr[dev]);
      g_ws_ptr[dev] = nullptr;
      g_ws_bytes[dev] = 0;
      g_ws_in_graph[dev] = false;
      if (e != cudaSuccess) return cuda_fail(e, "cudaFree(workspace)");
    }
    const size_t want = align_up(bytes < (1u << 20) ? (1u << 20) : bytes, 1u << 20);
    e = cudaMalloc(&g_ws_ptr[dev], want);
    if (e != cudaSuccess) {
      g_ws_ptr[dev] = nullptr;
      return cuda_fail(e, "cudaMalloc(workspace)");
    }
    g_ws_bytes[dev] = want;
  }
  if (g_cnt_bytes[dev] < counter_bytes) {
    if (g_cnt_ptr[dev] != nullptr) {
      e = g_cnt_in_graph[dev] ? cudaSuccess : cudaFree(g_cnt_ptr[dev]);
      g_cnt_ptr[dev] = nullptr;
      g_cnt_bytes[dev] = 0;
      g_cnt_in_graph[dev] = false;
      if (e != cudaSuccess) return cuda_fail(e, "cudaFree(tickets)");
    }
    const size_t want = align_up(counter_bytes < 65536 ? 65536 : counter_bytes, 65536);
    void* p = nullptr;
    e = cudaMalloc(&p, want);
    if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc(tickets)");
    // Merge tickets start at zero; every decode leaves them zero, a timed-out one too.
    e = cudaMemset(p, 0, want);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
      cudaFree(p);
      return cuda_fail(e, "cudaMemset(tickets)");
    }
    g_cnt_ptr[dev] = p;
    g_cnt_bytes[dev] = want;
  }
  if (status != cudaStreamCaptureStatusNone) g_ws_in_graph[dev] = g_cnt_in_graph[dev] = true;
  *ptr = g_ws_ptr[dev];
  *counters = static_cast<int32_t*>(g_cnt_ptr[dev]);
  return PA_OK;
}

int raise_smem_limit(const void* kernel, int bytes, int device, RaisedDevices* raised) {
  const uint64_t bit = 1ull << (device & 63);
  if (raised->done.load(std::memory_order_acquire) & bit) return PA_OK;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(shared memory)");
  raised->done.fetch_or(bit, std::memory_order_release);
  return PA_OK;
}

int ScratchHold::of_stream(size_t bytes, void* stream, void** ptr, size_t ticket_bytes, int32_t** tickets) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(static_cast<cudaStream_t>(stream), &status);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamIsCapturing");
  if (status != cudaStreamCaptureStatusNone)
    return fail(PA_ERR_INVALID_ARG, "a captured call needs a workspace of the caller's");
  unsigned long long id = 0;
  e = cudaStreamGetId(static_cast<cudaStream_t>(stream), &id);
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamGetId");
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  lock_ = std::unique_lock<std::mutex>(g_scratch_mutex);
  KeptScratch* mine = &g_kept[dev][0];  // the stream's, or the one not used for longest
  for (KeptScratch& k : g_kept[dev]) {
    if (k.used != 0 && k.stream == id) {
      mine = &k;
      break;
    }
    if (k.used < mine->used) mine = &k;
  }
  const bool held = mine->used != 0 && mine->stream == id;
  if (mine->bytes < bytes || mine->ticket_bytes < ticket_bytes || !held) {
    if (mine->used != 0) {  // calls that use the buffer may still run
      e = cudaDeviceSynchronize();
      if (e != cudaSuccess) return cuda_fail(e, "cudaDeviceSynchronize(scratch)");
    }
    if (mine->bytes < bytes) {
      size_t want = (size_t)16 << 20;
      while (want < bytes) want *= 2;
      if (mine->ptr != nullptr) (void)cudaFree(mine->ptr);
      mine->ptr = nullptr;
      mine->bytes = 0;
      mine->used = 0;
      e = cudaMalloc(&mine->ptr, want);
      if (e != cudaSuccess) {
        mine->ptr = nullptr;
        return cuda_fail(e, "cudaMalloc(scratch)");
      }
      mine->bytes = want;
    }
    if (mine->ticket_bytes < ticket_bytes) {
      const size_t want = align_up(ticket_bytes < 65536 ? 65536 : ticket_bytes, 65536);
      if (mine->tickets != nullptr) (void)cudaFree(mine->tickets);
      mine->tickets = nullptr;
      mine->ticket_bytes = 0;
      mine->used = 0;
      void* p = nullptr;
      e = cudaMalloc(&p, want);
      if (e != cudaSuccess) return cuda_fail(e, "cudaMalloc(tickets)");
      e = cudaMemset(p, 0, want);
      if (e == cudaSuccess) e = cudaDeviceSynchronize();
      if (e != cudaSuccess) {
        cudaFree(p);
        return cuda_fail(e, "cudaMemset(tickets)");
      }
      mine->tickets = p;
      mine->ticket_bytes = want;
    }
    mine->stream = id;
  }
  mine->used = ++g_kept_calls;
  *ptr = mine->ptr;
  if (tickets != nullptr) *tickets = static_cast<int32_t*>(mine->tickets);
  return PA_OK;
}

void take_wait_test(long long* stall_tile, unsigned long long* wait_limit_ns) {
  *stall_tile = g_stall_tile;
  *wait_limit_ns = g_stall_limit_us ? 1000ull * g_stall_limit_us : 2000000000ull;
  g_stall_tile = -1;
  g_stall_limit_us = 0;
}

}  // namespace pa

extern "C" int pa_test_stall_copy(long long tile, unsigned int wait_limit_us) {
  pa::clear_error();
  if (tile < -1) return pa::fail(PA_ERR_INVALID_ARG, "pa_test_stall_copy: tile %lld < -1", tile);
  pa::g_stall_tile = tile;
  pa::g_stall_limit_us = tile < 0 ? 0u : wait_limit_us;
  return PA_OK;
}

extern "C" const char* pa_last_error(void) { return pa::g_message; }

extern "C" int pa_version(void) { return 100; }
