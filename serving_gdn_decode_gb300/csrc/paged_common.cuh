// Launches of the full-attention operators, and their failure word.
//
// Launches.  The kernels of a decode step are short, so each is launched with
// programmatic stream serialization: it may be set up while the kernel before
// it on the stream still runs, and begins with begin_in_order(), which waits
// for that kernel's end (and so for its memory) before anything is read.
// The order on the stream is that of plain launches.
//
// The failure word of one translation unit's kernels (one word per device, a
// module global), as the chunked kernels have: bits are the GDN_DEVICE_* of
// gdn.h, set by a kernel that met data it cannot follow.
#pragma once

#include <cuda_runtime.h>

namespace gdn {
namespace {

__device__ unsigned int g_paged_status = 0u;

__device__ __forceinline__ void begin_in_order() {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_in_order(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

__device__ __forceinline__ void report(unsigned int bits) { atomicOr(&g_paged_status, bits); }

// Host: the word's address on the current device.
inline cudaError_t paged_status_word(unsigned int **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_paged_status);
}

}  // namespace
}  // namespace gdn
