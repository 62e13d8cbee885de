// Host-side helpers of the C ABI's entry points: device properties, argument checks and the
// optional per-kernel trace (one trace for the whole library).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <mutex>

#include "mok.h"

namespace mok_api {

constexpr int kMaxDevices = 64;

inline int sm_count() {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev] = n;
  }
  return cache[dev];
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

#define MOK_CUDA(call)                       \
  do {                                       \
    if ((call) != cudaSuccess) return MOK_ERR_CUDA; \
  } while (0)

// ------------------------------------------------------------------ per-kernel trace
struct TraceRec {
  const char* name;
  cudaEvent_t start, stop;
};

struct Trace {
  std::mutex mu;
  bool on = false;
  int cap = 0;
  int used = 0;
  TraceRec* recs = nullptr;
};
inline Trace g_trace;

// Records a start event before and a stop event after the launch `call` on stream `st`.
template <typename F>
cudaError_t traced(const char* name, cudaStream_t st, F&& call) {
  TraceRec* rec = nullptr;
  if (g_trace.on) {
    std::lock_guard<std::mutex> lock(g_trace.mu);
    if (g_trace.on && g_trace.used < g_trace.cap) {
      rec = &g_trace.recs[g_trace.used++];
      rec->name = name;
    }
  }
  if (rec) cudaEventRecord(rec->start, st);
  const cudaError_t err = call();
  if (rec) cudaEventRecord(rec->stop, st);
  return err;
}

#define MOK_LAUNCH(name, st, expr) MOK_CUDA(mok_api::traced(name, st, [&] { return (expr); }))

}  // namespace mok_api
