// Rotary positions with several axes on q and k, with the store of k and v in
// the paged cache (gdn_rope, gdn_rope_store).
//
// Pair j of a head, elements (a, b) = (x[j], x[j + R/2]), or (x[2j], x[2j+1])
// interleaved, at the token's position p on the pair's axis:
//     (a, b) -> (a c - b s, b c + a s),  c = cos_sin[p][j], s = cos_sin[p][R/2 + j]
// with -s for the inverse, which is the transpose and so the gradient's map.
// Products and sums are f32; a result is rounded once, when stored.
//
// One pass: every element is read once and written once, so HBM bounds long
// prompts and latency bounds decode steps.  A CTA takes one token (or a part of
// its heads): the token's R cos/sin values are gathered once into shared memory
// for all heads, while the row data is already on its way into registers.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // items (two vectors each) a thread has in flight
constexpr int kMaxRot = 256;

// E contiguous elements: one 16-byte access, or a single element.
template <typename T, int E>
struct alignas(sizeof(T) * E) Vec {
  T x[E];
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float *d, float x) { *d = x; }
__device__ __forceinline__ void narrow(__nv_bfloat16 *d, float x) { *d = __float2bfloat16_rn(x); }

struct RopeDivs {
  FastDiv items, page;
};

template <typename T, int E>
__global__ void __launch_bounds__(kThreads) gdn_rope_kernel(const __grid_constant__ RopeArgs a,
                                                            const RopeDivs dv) {
  using V = Vec<T, E>;
  __shared__ float s_cs[kMaxRot];
  const gdn_rope_params &p = a.p;
  const uint32_t token = blockIdx.x, half = p.rot_dim / 2;
  const bool store = a.v != nullptr, inter = (p.flags & GDN_ROPE_INTERLEAVED) != 0;
  const uint32_t per_row = p.head_dim / (2 * E), rot_items = p.rot_dim / (2 * E);

  long long slot_at = -1;  // element offset of the token's slot in the caches
  if (store) {
    const int slot = a.slot_map[token];
    if (slot >= 0) {
      const uint32_t page = dv.page.div(static_cast<uint32_t>(slot));
      if (page < p.n_pages)
        slot_at = page * p.cache_page_stride + (slot - static_cast<long long>(page) * p.page_size) * p.cache_slot_stride;
      else if (threadIdx.x == 0)
        report(GDN_DEVICE_BAD_PAGE);
    }
  }
  // rows of the token: q heads, k heads, v heads; without a slot k and v go nowhere
  const uint32_t rows = p.n_q_heads + (store ? (slot_at >= 0 ? 2 * p.n_kv_heads : 0) : p.n_kv_heads);
  const uint32_t n_items = rows * per_row;

  bool staged = false;
  for (uint32_t i0 = blockIdx.y * (kThreads * kUnroll) + threadIdx.x; i0 < n_items || !staged;
       i0 += gridDim.y * (kThreads * kUnroll)) {
    V lo[kUnroll], hi[kUnroll];
    const T *src[kUnroll];
    T *dst[kUnroll];
    uint32_t col[kUnroll], gap[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t item = i0 + u * kThreads;
      if (item >= n_items) continue;
      const uint32_t row = dv.items.div(item), j = item - row * per_row;
      // the item's two vectors: a pair's two halves, or neighbours
      const bool split = !inter && j < rot_items;
      col[u] = split ? j * E : j * 2 * E;
      gap[u] = split ? half : E;
      if (row < p.n_q_heads) {
        src[u] = static_cast<const T *>(a.q) + token * p.q_stride + row * p.head_dim;
        dst[u] = static_cast<T *>(a.q_out) + token * p.q_out_stride + row * p.head_dim;
      } else if (row < p.n_q_heads + p.n_kv_heads) {
        const uint32_t h = row - p.n_q_heads;
        src[u] = static_cast<const T *>(a.k) + token * p.k_stride + h * p.head_dim;
        dst[u] = store ? static_cast<T *>(a.k_cache) + slot_at + h * p.cache_head_stride
                       : static_cast<T *>(a.k_out) + token * p.k_out_stride + h * p.head_dim;
      } else {
        const uint32_t h = row - p.n_q_heads - p.n_kv_heads;
        src[u] = static_cast<const T *>(a.v) + token * p.v_stride + h * p.head_dim;
        dst[u] = static_cast<T *>(a.v_cache) + slot_at + h * p.cache_head_stride;
        col[u] = j * 2 * E;
        gap[u] = E;
      }
      lo[u] = *reinterpret_cast<const V *>(src[u] + col[u]);
      hi[u] = *reinterpret_cast<const V *>(src[u] + col[u] + gap[u]);
    }
    if (!staged) {
      for (uint32_t j = threadIdx.x; j < half; j += kThreads) {
        const int pos = a.positions[p.axis_of_pair[j] * p.positions_stride + token];
        float c, s;
        if (static_cast<uint32_t>(pos) < p.n_positions) {
          const float *t = a.cos_sin + static_cast<uint64_t>(pos) * p.rot_dim;
          c = t[j];
          s = t[half + j];
        } else {  // no such row: the token's rotated values are NaN
          c = s = nanf("");
          report(GDN_DEVICE_BAD_POSITION);
        }
        s_cs[j] = c;
        s_cs[half + j] = (p.flags & GDN_ROPE_INVERSE) ? -s : s;
      }
      __syncthreads();
      staged = true;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const uint32_t item = i0 + u * kThreads;
      if (item >= n_items) continue;
      const uint32_t row = dv.items.div(item), j = item - row * per_row;
      if (row < p.n_q_heads + p.n_kv_heads && j < rot_items) {
        const uint32_t c0 = j * E;  // first of the item's E pairs
        if (inter) {
          if constexpr (E == 1) {  // the pair is (lo, hi)
            const float fa = widen(lo[u].x[0]), fb = widen(hi[u].x[0]), c = s_cs[c0], s = s_cs[half + c0];
            narrow(&lo[u].x[0], fa * c - fb * s);
            narrow(&hi[u].x[0], fb * c + fa * s);
          } else {
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
              const float c = s_cs[c0 + e], s = s_cs[half + c0 + e];
              const float c2 = s_cs[c0 + E / 2 + e], s2 = s_cs[half + c0 + E / 2 + e];
              const float fa = widen(lo[u].x[2 * e]), fb = widen(lo[u].x[2 * e + 1]);
              const float ga = widen(hi[u].x[2 * e]), gb = widen(hi[u].x[2 * e + 1]);
              narrow(&lo[u].x[2 * e], fa * c - fb * s);
              narrow(&lo[u].x[2 * e + 1], fb * c + fa * s);
              narrow(&hi[u].x[2 * e], ga * c2 - gb * s2);
              narrow(&hi[u].x[2 * e + 1], gb * c2 + ga * s2);
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float c = s_cs[c0 + e], s = s_cs[half + c0 + e];
            const float fa = widen(lo[u].x[e]), fb = widen(hi[u].x[e]);
            narrow(&lo[u].x[e], fa * c - fb * s);
            narrow(&hi[u].x[e], fb * c + fa * s);
          }
        }
      }
      *reinterpret_cast<V *>(dst[u] + col[u]) = lo[u];
      *reinterpret_cast<V *>(dst[u] + col[u] + gap[u]) = hi[u];
    }
  }
}

template <typename T, int E>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  const gdn_rope_params &p = a.p;
  const uint32_t per_row = p.head_dim / (2 * E);
  const uint32_t items = (p.n_q_heads + p.n_kv_heads * (a.v ? 2 : 1)) * per_row;
  const RopeDivs dv{FastDiv(per_row), FastDiv(p.page_size ? p.page_size : 1)};
  const uint32_t y = (items + kThreads * kUnroll - 1) / (kThreads * kUnroll);
  gdn_rope_kernel<T, E><<<dim3(p.n_tokens, y < 65535 ? y : 65535), kThreads, 0, stream>>>(a, dv);
  return cudaGetLastError();
}

// Whether every 16-byte vector of E elements that the vector form accesses is
// aligned and none crosses the rotated part's or a head's end.
template <typename T>
bool vectors_fit(const RopeArgs &a) {
  constexpr int E = 16 / sizeof(T);
  const gdn_rope_params &p = a.p;
  if (p.head_dim % (2 * E) || p.rot_dim % (2 * E)) return false;
  const void *ptrs[] = {a.q, a.k, a.v, a.q_out, a.k_out, a.k_cache, a.v_cache};
  for (const void *x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % 16) return false;
  const int64_t strides[] = {p.q_stride, p.k_stride, a.v ? p.v_stride : 0, p.q_out_stride,
                             a.k_out ? p.k_out_stride : 0, a.v ? p.cache_page_stride : 0,
                             a.v ? p.cache_head_stride : 0, a.v ? p.cache_slot_stride : 0};
  for (int64_t s : strides)
    if (s % E) return false;
  return true;
}

template <typename T>
cudaError_t launch_type(const RopeArgs &a, cudaStream_t stream) {
  return vectors_fit<T>(a) ? launch<T, 16 / sizeof(T)>(a, stream) : launch<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  return a.p.dtype == GDN_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<float>(a, stream);
}

cudaError_t rope_status(unsigned int *bits, bool reset, cudaStream_t stream) {
  return read_paged_status(bits, reset, stream);
}

}  // namespace gdn
