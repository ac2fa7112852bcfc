// workspace_cache.h -- the workspaces that the library keeps, one for each (device, stream) of a kind: found, or
// allocated on first use.  Host code only, so that a test can stand in for the runtime's calls.
#pragma once

#include <map>
#include <mutex>
#include <utility>

#include "qmv_internal.h"

namespace qmv {

using WorkspaceCache = std::map<std::pair<int, cudaStream_t>, Workspace>;

constexpr size_t kMaxWorkspaces = 64;  // of a kind

// Bytes of the counter region for n counters (a multiple of 256); carve `bytes` at `base`
// into n counters followed by the parts.
inline size_t workspace_counter_bytes(int n) { return ((size_t)n * sizeof(unsigned) + 255) / 256 * 256; }

inline void workspace_carve(void* base, size_t bytes, int n, Workspace* ws) {
  const size_t cb = workspace_counter_bytes(n);
  ws->counters = static_cast<unsigned*>(base);
  ws->max_counters = n;
  ws->partials = reinterpret_cast<float*>(static_cast<uint8_t*>(base) + cb);
  ws->max_partial_floats = bytes > cb ? (bytes - cb) / sizeof(float) : 0;
}

// The caller holds the cache's lock.  A failure is told by the return value alone: callers that carry on without a
// workspace return success, and an error left behind as the thread's last one would be taken for that of the next
// launch that somebody checks.
inline cudaError_t cached_workspace(WorkspaceCache& cache, int device, cudaStream_t stream, size_t bytes, int counters,
                                    Workspace* ws) {
  auto failed = [](cudaError_t err) {
    cudaGetLastError();
    return err;
  };
  const auto key = std::make_pair(device, stream);
  auto it = cache.find(key);
  if (it != cache.end()) {
    *ws = it->second;
    return cudaSuccess;
  }
  if (cache.size() >= kMaxWorkspaces) return cudaErrorMemoryAllocation;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  cudaError_t err = cudaStreamIsCapturing(stream, &cs);
  if (err != cudaSuccess) return failed(err);
  if (cs != cudaStreamCaptureStatusNone) return cudaErrorNotReady;  // no allocation while capturing
  void* base = nullptr;
  err = cudaMalloc(&base, bytes);
  if (err != cudaSuccess) return failed(err);
  err = cudaMemsetAsync(base, 0, workspace_counter_bytes(counters), stream);
  if (err != cudaSuccess) {
    cudaFree(base);
    return failed(err);
  }
  Workspace w;
  workspace_carve(base, bytes, counters, &w);
  try {
    cache.emplace(key, w);
  } catch (...) {  // nothing is thrown through the C entry points
    cudaFree(base);
    return cudaErrorMemoryAllocation;
  }
  *ws = w;
  return cudaSuccess;
}

}  // namespace qmv
