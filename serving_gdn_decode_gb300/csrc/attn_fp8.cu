// Attention of each request's newest tokens over its 8-bit paged cache
// (gdn_attn_paged_fp8): out = sum_j softmax_j(scale q.k_j) v_j, where an element
// of k_j and v_j is a code times the scale of its page and key head.
//
// The plain form of the kernel: a warp takes one query row and goes through its
// keys, an element of the head per lane, with the running maximum and sum.
#include <cuda_runtime.h>

#include "device_io.cuh"
#include "fp8_common.cuh"
#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;

template <typename T, int D>
__global__ void __launch_bounds__(128) gdn_attn_fp8_kernel(const __grid_constant__ AttnFp8Args a) {
  constexpr int E = D / 32;
  const gdn_attn_params &p = a.p;
  const int lane = threadIdx.x & 31;
  begin_in_order();
  const uint32_t s = blockIdx.x, head = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (head >= p.n_q_heads) return;
  const uint32_t kv_head = head / (p.n_q_heads / p.n_kv_heads);
  int t0 = s, t1 = s + 1;
  if (a.token_start) {
    t0 = a.token_start[s];
    t1 = a.token_start[s + 1];
  }
  const int n = static_cast<int>(p.n_tokens);
  bool bad = false;
  if (t0 < 0 || t1 < t0 || t1 > n) {
    bad = true;
    t0 = min(max(t0, 0), n);
    t1 = min(max(t1, t0), n);
  }
  int len = a.kv_lens[s];
  const long long most = static_cast<long long>(p.max_pages) * p.page_size;
  if (len < 0 || len > most) {
    bad = true;
    len = len < 0 ? 0 : static_cast<int>(most);
  }
  if (bad && lane == 0) report(GDN_DEVICE_BAD_REQUEST);
  // the keys that any of the request's rows sees: a page that is not there makes all of them NaN
  const long long first = p.window ? static_cast<long long>(len) - (t1 - t0) + 1 - p.window : 0;
  bool missing = false;
  if (t1 > t0 && len > 0)
    for (int64_t j = (first > 0 ? first : 0) / p.page_size + lane; j <= (len - 1) / static_cast<int>(p.page_size); j += 32)
      missing |= static_cast<uint32_t>(a.block_table[static_cast<uint64_t>(s) * p.max_pages + j]) >= p.n_pages;
  missing = __any_sync(kFull, missing);
  if (missing && lane == 0) report(GDN_DEVICE_BAD_PAGE);
  for (int t = t0; t < t1; ++t) {
    const int hi = len - (t1 - t) + 1;
    const long long lo = p.window ? max(0ll, static_cast<long long>(hi) - p.window) : 0;
    float q[E], acc[E] = {}, m = -3.402823466e38f, l = 0.0f;
    for (int e = 0; e < E; ++e) q[e] = Act<T>::get(static_cast<const T *>(a.q) + t * p.q_stride + head * D + lane * E + e);
    for (int j = static_cast<int>(lo); j < hi && !missing; ++j) {
      const uint32_t page = a.block_table[static_cast<uint64_t>(s) * p.max_pages + j / p.page_size];
      const int64_t at = page * p.cache_page_stride + kv_head * p.cache_head_stride + j % p.page_size * p.cache_slot_stride + lane * E;
      const float ks = a.k_scale[static_cast<uint64_t>(page) * p.n_kv_heads + kv_head];
      const float vs = a.v_scale[static_cast<uint64_t>(page) * p.n_kv_heads + kv_head];
      float x = 0.0f;
      for (int e = 0; e < E; ++e) x += q[e] * codes_f32x2(static_cast<const uint8_t *>(a.k_cache)[at + e], 0).x;
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(kFull, x, d);
      x *= p.scale * ks;
      const float top = fmaxf(m, x), f = expf(m - top), w = expf(x - top);
      m = top;
      l = l * f + w;
      for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + w * (vs * codes_f32x2(static_cast<const uint8_t *>(a.v_cache)[at + e], 0).x);
    }
    for (int e = 0; e < E; ++e)
      Act<T>::put(static_cast<T *>(a.output) + t * p.out_stride + head * D + lane * E + e,
                  missing ? __int_as_float(0x7fffffff) : hi <= 0 ? 0.0f : acc[e] / l);
  }
}

template <typename T>
cudaError_t launch(const AttnFp8Args &a, cudaStream_t stream) {
  const dim3 grid(a.p.n_seqs, (a.p.n_q_heads + 3) / 4);
  return a.p.head_dim == 64    ? launch_in_order(gdn_attn_fp8_kernel<T, 64>, grid, 128, 0, stream, a)
         : a.p.head_dim == 128 ? launch_in_order(gdn_attn_fp8_kernel<T, 128>, grid, 128, 0, stream, a)
                               : launch_in_order(gdn_attn_fp8_kernel<T, 256>, grid, 128, 0, stream, a);
}

}  // namespace

size_t attn_fp8_workspace_bytes(const gdn_attn_params &) { return 16; }

cudaError_t launch_attn_paged_fp8(const AttnFp8Args &a, cudaStream_t stream) {
  return a.p.dtype == GDN_DTYPE_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

cudaError_t attn_fp8_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
