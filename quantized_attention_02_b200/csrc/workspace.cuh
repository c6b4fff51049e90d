// workspace.cuh -- stream-ordered device workspace for the entry points that need one: the forward passes, the
// preparation steps and the joined parts of the paged and the cross attention.
//
// Allocations come from a memory pool owned by the library (one per device, created on first
// use), not from the process's default pool, whose settings belong to the application.  The
// pool's release threshold is unlimited: memory freed by a call stays reserved for the next
// call instead of being handed back to the driver at every synchronization, which would make
// the first call after each synchronize map the workspace again (measured: 2-15 ms of host
// time for that call).  The pool therefore keeps the largest workspace used so far reserved
// until the process exits.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstddef>

namespace sage {

// cudaMallocFromPoolAsync on the library's pool of the current device; returns the CUDA
// error (cudaSuccess on success).  Free with cudaFreeAsync on a stream ordered after the uses.
cudaError_t workspace_alloc(void** p, size_t bytes, cudaStream_t st);

// cudaFuncAttributeMaxDynamicSharedMemorySize of a kernel on the current device, once per device: `done` (one per
// kernel) has a bit for each device it was set on.  Setting it twice from two threads is harmless.
inline cudaError_t allow_shared_memory(std::atomic<unsigned long long>& done, const void* kernel, int bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace sage
