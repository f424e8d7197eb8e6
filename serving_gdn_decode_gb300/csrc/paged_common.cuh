// The failure word of one translation unit's kernels (one word per device, a
// module global), as the chunked kernels have: bits are the GDN_DEVICE_* of
// gdn.h, set by a kernel that met data it cannot follow.
#pragma once

#include <cuda_runtime.h>

namespace gdn {
namespace {

__device__ unsigned int g_paged_status = 0u;

__device__ __forceinline__ void report(unsigned int bits) { atomicOr(&g_paged_status, bits); }

// Host: *bits = this translation unit's word after all work on `stream` so
// far; cleared afterwards when `reset`.  Symbol copies only; synchronises.
inline cudaError_t read_paged_status(unsigned int *bits, bool reset, cudaStream_t stream) {
  unsigned int h = 0u;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&h, g_paged_status, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess && reset) {
    static const unsigned int zero = 0u;
    e = cudaMemcpyToSymbolAsync(g_paged_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, stream);
  }
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  *bits = e == cudaSuccess ? h : 0u;
  return e;
}

}  // namespace
}  // namespace gdn
