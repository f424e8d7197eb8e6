// Internal interface between the C-ABI host code (paged_abi.cu) and the
// launchers of the full-attention operators: kv_plan.cu, rope.cu, attn_paged.cu,
// kv_fp8.cu, attn_fp8.cu.
// Nothing here is exported from the shared library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdn.h"

namespace gdn {

// Unsigned division by a constant of the call, for dividends below 2^31:
// n / d = (mulhi(n, m) + n) >> s with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1 (the round-up method of Granlund and
// Montgomery, "Division by invariant integers using multiplication", 1994).
struct FastDiv {
  uint32_t d, m, s;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), m(0), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
#endif
};

struct PlanArgs {
  const int32_t *ctx_lens, *new_lens, *owned, *free_pages, *n_free;
  int32_t *block_table, *kv_lens, *owned_out, *n_free_out, *token_start, *slot_map, *positions;
  gdn_kv_plan_params p;
};
cudaError_t launch_kv_plan(const PlanArgs &a, cudaStream_t stream);

struct RopeArgs {
  const void *q, *k, *v;  // v == nullptr: no cache
  const int32_t *positions, *slot_map;
  const float *cos_sin;
  void *q_out, *k_out;      // k_out == nullptr: k goes to the cache
  void *k_cache, *v_cache;
  gdn_rope_params p;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream);

struct AttnArgs {
  const void *q, *k_cache, *v_cache;
  const int32_t *block_table, *kv_lens, *token_start;
  void *output;
  gdn_attn_params p;
  void *workspace;
};
size_t attn_workspace_bytes(const gdn_attn_params &p);
cudaError_t launch_attn_paged(const AttnArgs &a, cudaStream_t stream);

struct KvFp8Args {
  const void *k, *v;  // store: the rows to store; load: nullptr
  void *k_out, *v_out;  // load: the rows to write; store: nullptr
  const int32_t *slot_map;
  void *k_cache, *v_cache;
  float *k_scale, *v_scale;
  gdn_kv_fp8_params p;
};
cudaError_t launch_kv_store_fp8(const KvFp8Args &a, cudaStream_t stream);
cudaError_t launch_kv_load_fp8(const KvFp8Args &a, cudaStream_t stream);

struct AttnFp8Args {
  const void *q, *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *kv_lens, *token_start;
  void *output;
  gdn_attn_params p;
  void *workspace;
};
size_t attn_fp8_workspace_bytes(const gdn_attn_params &p);
cudaError_t launch_attn_paged_fp8(const AttnFp8Args &a, cudaStream_t stream);
void attn_fp8_wait_clocks(uint32_t clocks);  // 0: the default

// The status words of the files' kernels on the current device (read_device_status).
cudaError_t kv_plan_status_word(unsigned int **word);
cudaError_t rope_status_word(unsigned int **word);
cudaError_t attn_paged_status_word(unsigned int **word);
cudaError_t kv_fp8_status_word(unsigned int **word);
cudaError_t attn_fp8_status_word(unsigned int **word);

}  // namespace gdn
