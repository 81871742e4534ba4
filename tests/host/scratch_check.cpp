// Host check of the library's own scratch (pa_host.cu against a stand-in for the CUDA
// runtime) under calls from several threads: from the lookup of a call's buffer to its
// last launch no other thread frees it, gives it to another stream or queues launches
// of its own on it, and a buffer changes hands only when the device is done with it.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>
#include <chrono>
#include <map>
#include <mutex>
#include <thread>
#include <vector>

#include "pa_internal.h"

struct Use {
  unsigned long long stream = 0;
  int call = 0;      // the call between its lookup and its last launch, 0: none
  bool pending = false;  // launches queued since the device was synchronised
};
static std::mutex fake;
static std::map<void*, Use> memory;
static std::atomic<int> faults{0}, syncs{0};
static void fault(const char* what) {
  if (faults++ == 0) printf("%s\n", what);
}

const char* cudaGetErrorString(cudaError_t) { return ""; }
const char* cudaGetErrorName(cudaError_t) { return ""; }
cudaError_t cudaGetDevice(int* d) { return *d = 0, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrComputeCapabilityMajor ? 10 : a == cudaDevAttrComputeCapabilityMinor ? 3 : 152;
  return cudaSuccess;
}
cudaError_t cudaMalloc(void** p, size_t n) {
  std::lock_guard<std::mutex> l(fake);
  *p = malloc(n < 64 ? 64 : 64 + n % 64);  // the address is all that matters
  memory[*p] = Use{};
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {  // waits for the device, as the runtime's does
  cudaDeviceSynchronize();
  std::lock_guard<std::mutex> l(fake);
  if (memory.count(p) == 0) fault("freed twice");
  if (memory[p].call != 0) fault("freed between a call's lookup and its last launch");
  memory.erase(p);
  return cudaSuccess;  // (not given back to malloc: no address is used twice)
}
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaDeviceSynchronize() {
  std::lock_guard<std::mutex> l(fake);
  ++syncs;
  for (auto& m : memory) m.second.pending = false;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t s, cudaStreamCaptureStatus* st) {
  *st = (uintptr_t)s == 99 ? cudaStreamCaptureStatusActive : cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaStreamGetId(cudaStream_t s, unsigned long long* id) { return *id = (uintptr_t)s + 1, cudaSuccess; }

// A call of three launches on its buffer.
static void call(int id, unsigned long long stream, size_t bytes, bool plain) {
  pa::ScratchHold hold;
  void* p = nullptr;
  int32_t* tickets = nullptr;
  const int rc = plain ? hold.plain(bytes, 1024, (void*)stream, &p, &tickets) : hold.of_stream(bytes, (void*)stream, &p);
  if (rc != 0) return fault("no scratch");
  for (int launch = 0; launch < 3; ++launch) {
    {
      std::lock_guard<std::mutex> l(fake);
      auto m = memory.find(p);
      if (m == memory.end()) return fault("launched on freed memory");
      if (launch > 0 && m->second.call != id) fault("launches of two calls mixed");
      if (!plain && m->second.pending && m->second.stream != stream) fault("two streams in one buffer");
      m->second = Use{stream, id, true};
    }
    std::this_thread::sleep_for(std::chrono::microseconds(20 * (id % 5)));
  }
  std::lock_guard<std::mutex> l(fake);
  if (memory.count(p)) memory[p].call = 0;
}

static void threads(int n, bool one_stream, bool plain, bool growing) {
  std::atomic<int> next{1};
  std::vector<std::thread> ts;
  for (int t = 0; t < n; ++t)
    ts.emplace_back([&, t] {
      for (int i = 0; i < 60; ++i)
        call(next++, one_stream ? 7 : (t * 5 + i) % 11, growing ? ((size_t)1 << 20) * (1 + (i * 7 + t) % 90) : 1000, plain);
    });
  for (auto& t : ts) t.join();
}

int main() {
  threads(2, true, false, false);
  threads(4, true, false, true);
  threads(4, false, false, true);  // eleven streams, eight buffers
  threads(4, true, true, true);
  {
    pa::ScratchHold hold;
    void* p = nullptr;
    if (hold.of_stream(64, (void*)99, &p) == 0) fault("given to a stream under capture");
  }
  {  // what a captured call has taken stays, however the scratch grows
    void *p = nullptr, *q = nullptr;
    int32_t *tickets = nullptr, *more = nullptr;
    {
      pa::ScratchHold hold;
      hold.plain(1000, 1000, (void*)99, &p, &tickets);
    }
    {
      pa::ScratchHold hold;
      hold.plain((size_t)1 << 30, (size_t)1 << 20, (void*)7, &q, &more);
    }
    if (p == q || tickets == more) fault("not grown");
    if (memory.count(p) == 0 || memory.count(tickets) == 0) fault("freed under a graph");
    {
      pa::ScratchHold hold;
      hold.plain((size_t)2 << 30, (size_t)2 << 20, (void*)7, &p, &tickets);
    }
    if (memory.count(q) != 0 || memory.count(more) != 0) fault("kept without a graph");
  }
  if (faults) return 1;
  printf("ok, %d times synchronised\n", (int)syncs);
  return 0;
}
