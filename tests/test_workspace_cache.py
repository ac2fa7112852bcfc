"""The kept workspaces (csrc/workspace_cache.h) on the host, with fakes of the runtime's calls: a call that does without a
workspace leaves no error behind."""
import os
import subprocess

from block_quantized_weight_q4_gb300.build import CSRC, nvcc

SOURCE = r"""
#include <cstdio>
#include <cstdlib>
#include "workspace_cache.h"

// Fakes: each call gives the error it was set to, which is then the last error, as in the runtime.
static cudaError_t last = cudaSuccess, malloc_gives = cudaSuccess, memset_gives = cudaSuccess, capturing_gives = cudaSuccess;
static cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
static int mallocs = 0, frees = 0;
static cudaError_t gives(cudaError_t e) { if (e != cudaSuccess) last = e; return e; }
extern "C" {
cudaError_t cudaGetLastError(void) { const cudaError_t e = last; last = cudaSuccess; return e; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* s) { *s = capture; return gives(capturing_gives); }
cudaError_t cudaMalloc(void** p, size_t n) {
  ++mallocs;
  if (malloc_gives == cudaSuccess) *p = std::malloc(n);
  return gives(malloc_gives);
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return gives(memset_gives); }
cudaError_t cudaFree(void* p) { ++frees; std::free(p); return cudaSuccess; }
}

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  qmv::WorkspaceCache cache;
  qmv::Workspace w{};
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(0x10);
  auto get = [&] { return qmv::cached_workspace(cache, 0, s, 1 << 16, 1024, &w); };
  malloc_gives = cudaErrorMemoryAllocation;
  CHECK(get() == cudaErrorMemoryAllocation && last == cudaSuccess && cache.empty());
  malloc_gives = cudaSuccess;
  memset_gives = cudaErrorInvalidValue;
  CHECK(get() == cudaErrorInvalidValue && last == cudaSuccess && cache.empty() && frees == 1);
  memset_gives = cudaSuccess;
  capturing_gives = cudaErrorStreamCaptureImplicit;
  CHECK(get() == cudaErrorStreamCaptureImplicit && last == cudaSuccess && cache.empty());
  capturing_gives = cudaSuccess;
  capture = cudaStreamCaptureStatusActive;
  const int before = mallocs;
  CHECK(get() == cudaErrorNotReady && last == cudaSuccess && mallocs == before);
  capture = cudaStreamCaptureStatusNone;
  CHECK(get() == cudaSuccess && cache.size() == 1 && w.max_counters == 1024);
  CHECK(w.max_partial_floats == ((1u << 16) - 4096) / 4 && reinterpret_cast<char*>(w.partials) == reinterpret_cast<char*>(w.counters) + 4096);
  unsigned* const had = w.counters;
  malloc_gives = cudaErrorMemoryAllocation;
  CHECK(get() == cudaSuccess && w.counters == had);
  // an error that was there before is the caller's: finding a kept workspace does not touch it
  last = cudaErrorInvalidConfiguration;
  CHECK(get() == cudaSuccess && last == cudaErrorInvalidConfiguration);
  return 0;
}
"""


def test_failures_leave_no_error_behind(tmp_path):
    (tmp_path / "t.cpp").write_text(SOURCE)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    if not os.path.exists(os.path.join(cuda, "cuda_runtime.h")):
        cuda = "/usr/local/cuda/include"
    exe = str(tmp_path / "t")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", CSRC, "-I", cuda, str(tmp_path / "t.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
