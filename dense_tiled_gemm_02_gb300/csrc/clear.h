// clear.h -- zeroing of a handle's device memory at its creation.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <initializer_list>

namespace gb300 {

struct Clear {
  void* at;
  size_t bytes;
};

// Zeroes the ranges before it returns.  A plain cudaMemset would only be
// enqueued, on the null stream: a handle's first run on a non-blocking stream
// is not ordered after that, and could find its flags, or rows it had already
// copied into the workspace, cleared under it.
inline cudaError_t clear_now(std::initializer_list<Clear> ranges) {
  cudaStream_t st;
  cudaError_t e = cudaStreamCreateWithFlags(&st, cudaStreamNonBlocking);
  if (e != cudaSuccess) return e;
  for (const Clear& r : ranges)
    if (e == cudaSuccess && r.bytes) e = cudaMemsetAsync(r.at, 0, r.bytes, st);
  const cudaError_t done = cudaStreamSynchronize(st);
  cudaStreamDestroy(st);
  return e != cudaSuccess ? e : done;
}

}  // namespace gb300
