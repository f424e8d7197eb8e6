// The device status word (gdn_device_status): every file whose kernels can fail
// at run time has a word of its own; a small kernel takes them together, clearing
// them if asked in the same access, so that no bit set meanwhile is lost, and one
// copy brings the result.  One launch and one copy, however many files there are:
// a copy per file and one more to clear each, as they were, took 48 us, 86 us with
// the clearing, for five files; this takes 20 either way.
#include <cuda_runtime.h>

#include <mutex>

#include "gdn_internal.h"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr int kWords = 7;
struct Words {
  unsigned int *at[kWords];
};

__device__ unsigned int g_gathered;

__global__ void gdn_status_kernel(const Words w, bool reset) {
  unsigned int bits = 0;
#pragma unroll
  for (int i = 0; i < kWords; ++i) bits |= reset ? atomicExch(w.at[i], 0u) : atomicOr(w.at[i], 0u);
  g_gathered = bits;
}

}  // namespace

cudaError_t read_device_status(unsigned int *bits, bool reset, cudaStream_t stream) {
  static std::mutex one_at_a_time;  // g_gathered belongs to one call until it is copied
  *bits = 0;
  cudaError_t e = cudaStreamSynchronize(stream);  // the long wait, if any, outside the lock
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(one_at_a_time);
  Words w;
  cudaError_t (*const words[kWords])(unsigned int **) = {chunked_status_word, chunked_split_status_word, kv_plan_status_word,
                                                         rope_status_word, attn_paged_status_word, kv_fp8_status_word, attn_fp8_status_word};
  for (int i = 0; i < kWords; ++i)
    if ((e = words[i](&w.at[i])) != cudaSuccess) return e;
  gdn_status_kernel<<<1, 1, 0, stream>>>(w, reset);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  unsigned int h = 0;
  e = cudaMemcpyFromSymbolAsync(&h, g_gathered, sizeof h, 0, cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) *bits = h;
  return e;
}

}  // namespace gdn
