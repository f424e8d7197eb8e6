// The 8-bit paged cache: store of a step's k and v, and rows read back
// (gdn_kv_store_fp8, gdn_kv_load_fp8).
//
// A page holds e4m3 codes with one f32 scale per key head, for k and v apart: an
// element stands for code * scale.  The scale is the smallest power of two that
// keeps the page's largest magnitude within 448, e4m3's largest value.  e4m3 has
// its three mantissa bits at any magnitude, so a finer scale would not make the
// codes better, and a power of two makes the division exact, a code's value exact
// in bf16 and f32, and a page's codes easy to keep when a later token is larger:
// scaled down by a power of two they stay what they stand for, but for those that
// fall below the smallest codes.
//
// Store.  A unit of work is a run (neighbouring tokens of the call whose slots
// follow one another in a page) of one head of k or of v: its largest magnitude
// decides the scale, with the scale of the page's earlier tokens if it does not
// begin the page.  Units share nothing, so nothing is atomic.  A team of warps
// takes a unit and keeps its rows in registers between the maximum and the codes.
#include <cuda_runtime.h>

#include "fp8_common.cuh"
#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kLeast = -110, kMost = 119;  // exponents of a scale: code * scale stays a normal, finite f32 and bf16
constexpr int kKeep = 8;                   // vectors of a unit that a lane keeps

// 16 bytes of activations.
template <typename T>
struct Row16;
template <>
struct Row16<float> {
  static constexpr int kElems = 4;
  float4 x;
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w; }
  __device__ __forceinline__ void put(const float (&f)[4]) { x = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Row16<__nv_bfloat16> {
  static constexpr int kElems = 8;
  uint4 x;
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const unsigned w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void put(const float (&f)[8]) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned *>(&h);
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// A vector of E elements at p, which may be aligned to an element only.
template <typename T>
__device__ __forceinline__ Row16<T> load_row(const T *p, bool wide) {
  Row16<T> r;
  if (wide) {
    r.x = *reinterpret_cast<const decltype(r.x) *>(p);
  } else {
    T *e = reinterpret_cast<T *>(&r.x);
#pragma unroll
    for (int i = 0; i < Row16<T>::kElems; ++i) e[i] = p[i];
  }
  return r;
}
template <typename T>
__device__ __forceinline__ void store_row(T *p, const Row16<T> &r, bool wide) {
  if (wide) {
    *reinterpret_cast<decltype(r.x) *>(p) = r.x;
  } else {
    const T *e = reinterpret_cast<const T *>(&r.x);
#pragma unroll
    for (int i = 0; i < Row16<T>::kElems; ++i) p[i] = e[i];
  }
}

// The smallest power of two s with amax <= 448 s = 1.75 * 2^8 s, within the exponents' range.
__device__ __forceinline__ float least_scale(float amax) {
  const int bits = __float_as_int(amax);
  int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000);
  e = min(max(e, kLeast), kMost);
  return __int_as_float((e + 127) << 23);
}

struct StoreCall {
  KvFp8Args a;
  FastDiv page_div, row_div;  // by the page size; by the vectors of a row
  uint32_t row_vecs;
  uint32_t window;   // tokens whose runs' beginnings a team looks for
  uint32_t windows;
  bool wide;         // rows of k and v are aligned to 16 bytes
};

template <typename T, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128) gdn_kv_store_kernel(const __grid_constant__ StoreCall c) {
  constexpr int E = Row16<T>::kElems, kTeams = W > 4 ? 1 : 4 / W;  // of a CTA
  __shared__ float s_top[kTeams][W];
  const gdn_kv_fp8_params &p = c.a.p;
  const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * W), me = threadIdx.x % (32 * W);
  auto meet = [&] {
    if constexpr (W == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;\n" ::"r"(1 + team), "n"(32 * W) : "memory");
  };
  begin_in_order();
  const uint32_t unit = blockIdx.x * kTeams + team, which = blockIdx.y & 1, head = blockIdx.y >> 1;
  if (unit >= c.windows) return;  // the whole team
  const int n = static_cast<int>(p.n_tokens), t0 = unit * c.window, t1 = min(n, t0 + static_cast<int>(c.window));
  const T *src = static_cast<const T *>(which ? c.a.v : c.a.k) + head * p.head_dim;
  const int64_t src_stride = which ? p.v_stride : p.k_stride;
  uint8_t *cache = static_cast<uint8_t *>(which ? c.a.v_cache : c.a.k_cache) + head * p.cache_head_stride;
  float *scales = (which ? c.a.v_scale : c.a.k_scale) + head;
  const int32_t *slots = c.a.slot_map;

  for (int base = t0; base < t1; base += 32) {
    // the tokens at which runs begin
    const int i = base + lane;
    bool begins = false;
    if (i < t1) {
      const int slot = slots[i], before = i ? slots[i - 1] : -1;
      if (slot >= 0) {
        const uint32_t page = c.page_div.div(slot);
        const bool same = before >= 0 && c.page_div.div(before) == page;
        begins = !(same && before + 1 == slot);
        if (page >= p.n_pages) {
          if (begins) report(GDN_DEVICE_BAD_PAGE);
          begins = false;
        } else if (begins && same) {  // a page's tokens out of order
          report(GDN_DEVICE_BAD_REQUEST);
          begins = false;
        }
      }
    }
    for (unsigned left = __ballot_sync(kFull, begins); left; left &= left - 1) {
      const int first = base + __ffs(left) - 1;
      const int slot = slots[first];
      const uint32_t page = c.page_div.div(slot);
      const int place = slot - static_cast<int>(page * p.page_size), most = static_cast<int>(p.page_size) - place;
      int len = 1;  // tokens of the run
      for (bool go = true; go && len < most;) {
        const int j = len + lane;
        const unsigned ends = __ballot_sync(kFull, j >= most || first + j >= n || slots[first + j] != slot + j);
        len += ends ? __ffs(ends) - 1 : 32;
        go = ends == 0;
      }
      float *scale_at = scales + static_cast<uint64_t>(page) * p.n_kv_heads;
      const float old = place ? *scale_at : 0.0f;
      uint8_t *rows = cache + page * p.cache_page_stride;
      const int vecs = len * static_cast<int>(c.row_vecs);
      // the largest magnitude
      Row16<T> keep[kKeep];
      float top = 0.0f;
      auto at = [&](int x) {
        const int r = c.row_div.div(x);
        return src + (first + r) * src_stride + (x - r * static_cast<int>(c.row_vecs)) * E;
      };
      auto raise = [&](const Row16<T> &v) {
        float f[E];
        v.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float m = fabsf(f[e]);
          top = m <= 3.402823466e38f ? fmaxf(top, m) : top;
        }
      };
#pragma unroll
      for (int u = 0; u < kKeep; ++u) {
        const int x = u * 32 * W + me;
        if (x < vecs) keep[u] = load_row(at(x), c.wide);
      }
#pragma unroll
      for (int u = 0; u < kKeep; ++u)
        if (u * 32 * W + me < vecs) raise(keep[u]);
      for (int x = kKeep * 32 * W + me; x < vecs; x += 32 * W) raise(load_row(at(x), c.wide));
#pragma unroll
      for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
      if constexpr (W > 1) {
        if (lane == 0) s_top[team][me / 32] = top;
        meet();
#pragma unroll
        for (int w = 0; w < W; ++w) top = fmaxf(top, s_top[team][w]);
      }
      const float need = least_scale(top);
      const float scale = old > need && old <= 3.402823466e38f ? old : need, inv = 1.0f / scale;
      // the page's earlier tokens, on the new scale; those of a scale that is none (negative, infinite, NaN) are NaN
      if (place && scale != old) {
        const float by = old >= 0.0f && old <= 3.402823466e38f ? old * inv : __int_as_float(0x7fffffff);
        const int row16 = p.head_dim / 16, all = place * row16;
        for (int x = me; x < all; x += 32 * W) {
          uint4 *q = reinterpret_cast<uint4 *>(rows + x / row16 * p.cache_slot_stride + x % row16 * 16);
          uint4 y = *q;
          unsigned *w = &y.x;
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const float2 a = codes_f32x2(w[i4], 0), b = codes_f32x2(w[i4], 2);
            w[i4] = codes_of(a.x * by, a.y * by, b.x * by, b.y * by);
          }
          *q = y;
        }
      }
      auto put = [&](const Row16<T> &v, int x) {
        float f[E];
        v.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = fabsf(f[e]) <= 3.402823466e38f ? f[e] * inv : __int_as_float(0x7fffffff);
        const int r = c.row_div.div(x);
        uint8_t *to = rows + (place + r) * p.cache_slot_stride + (x - r * static_cast<int>(c.row_vecs)) * E;
        if constexpr (E == 8)
          *reinterpret_cast<uint2 *>(to) = make_uint2(codes_of(f[0], f[1], f[2], f[3]), codes_of(f[4], f[5], f[6], f[7]));
        else
          *reinterpret_cast<unsigned *>(to) = codes_of(f[0], f[1], f[2], f[3]);
      };
#pragma unroll
      for (int u = 0; u < kKeep; ++u) {
        const int x = u * 32 * W + me;
        if (x < vecs) put(keep[u], x);
      }
      for (int x = kKeep * 32 * W + me; x < vecs; x += 32 * W) put(load_row(at(x), c.wide), x);
      meet();  // s_top and the old scale have been read
      if (me == 0) *scale_at = scale;
    }
  }
}

// Rows read back: a warp takes a token's k and v, a lane E codes at a time, which are 16 bytes of the output.
struct LoadCall {
  KvFp8Args a;
  FastDiv page_div, row_div;
  uint32_t row_vecs, vecs;  // of a head's row; of a token's k
  bool wide;
};

template <typename T>
__global__ void __launch_bounds__(128) gdn_kv_load_kernel(const __grid_constant__ LoadCall c) {
  constexpr int E = Row16<T>::kElems, U = 4;
  const gdn_kv_fp8_params &p = c.a.p;
  const uint32_t lane = threadIdx.x & 31, token = blockIdx.x * 4 + (threadIdx.x >> 5);
  begin_in_order();
  if (token >= p.n_tokens) return;
  const int slot = c.a.slot_map[token];
  if (slot < 0) return;
  const uint32_t page = c.page_div.div(slot);
  const bool none = page >= p.n_pages;  // such rows are NaN
  if (none && lane == 0) report(GDN_DEVICE_BAD_PAGE);
  const int64_t row = none ? 0 : page * p.cache_page_stride + static_cast<int64_t>(slot - page * p.page_size) * p.cache_slot_stride;
  for (uint32_t x0 = 0; x0 < 2 * c.vecs; x0 += 32 * U) {
    uint2 codes[U];
    float scale[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t x = x0 + u * 32 + lane;
      if (x >= 2 * c.vecs) continue;
      const bool value = x >= c.vecs;
      const uint32_t y = value ? x - c.vecs : x, head = c.row_div.div(y), col = (y - head * c.row_vecs) * E;
      const uint8_t *q = static_cast<const uint8_t *>(value ? c.a.v_cache : c.a.k_cache) + row + head * p.cache_head_stride + col;
      if constexpr (E == 8) codes[u] = *reinterpret_cast<const uint2 *>(q);
      else codes[u].x = *reinterpret_cast<const unsigned *>(q);
      scale[u] = none ? __int_as_float(0x7fffffff) : (value ? c.a.v_scale : c.a.k_scale)[static_cast<uint64_t>(page) * p.n_kv_heads + head];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t x = x0 + u * 32 + lane;
      if (x >= 2 * c.vecs) continue;
      const bool value = x >= c.vecs;
      const uint32_t y = value ? x - c.vecs : x;
      float f[E];
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 g = codes_f32x2(e < 4 ? codes[u].x : codes[u].y, e & 2);
        f[e] = g.x * scale[u];
        f[e + 1] = g.y * scale[u];
      }
      Row16<T> r;
      r.put(f);
      T *to = (value ? static_cast<T *>(c.a.v_out) + token * p.v_stride : static_cast<T *>(c.a.k_out) + token * p.k_stride) +
              static_cast<uint64_t>(y) * E;
      store_row(to, r, c.wide);
    }
  }
}

// ------------------------------------------------------------ host

bool rows_wide(const KvFp8Args &a, uint32_t elems) {
  const void *ptrs[] = {a.k, a.v, a.k_out, a.v_out};
  for (const void *x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % 16) return false;
  return a.p.k_stride % elems == 0 && a.p.v_stride % elems == 0;
}

template <typename T, int W>
cudaError_t launch_store(StoreCall c, cudaStream_t stream) {
  const gdn_kv_fp8_params &p = c.a.p;
  constexpr uint32_t kTeams = W > 4 ? 1 : 4 / W;
  // With few tokens a team each; with many a page of them, so that hardly a team finds no run's beginning.
  const uint64_t units = static_cast<uint64_t>(p.n_tokens) * p.n_kv_heads * 2, enough = 152 * 32 / W;
  c.window = static_cast<uint32_t>(units / enough);
  if (c.window < 1) c.window = 1;
  if (c.window > p.page_size) c.window = p.page_size;
  c.windows = (p.n_tokens + c.window - 1) / c.window;
  return launch_in_order(gdn_kv_store_kernel<T, W>, dim3((c.windows + kTeams - 1) / kTeams, 2 * p.n_kv_heads), W > 4 ? 32 * W : 128, 0, stream, c);
}

template <typename T>
cudaError_t launch_store(const KvFp8Args &a, cudaStream_t stream) {
  constexpr uint32_t E = Row16<T>::kElems;
  StoreCall c;
  c.a = a;
  c.page_div = FastDiv(a.p.page_size);
  c.row_vecs = a.p.head_dim / E;
  c.row_div = FastDiv(c.row_vecs);
  c.wide = rows_wide(a, E);
  // warps enough for the longest run's rows to stay in registers
  const uint64_t rows = a.p.page_size < a.p.n_tokens ? a.p.page_size : a.p.n_tokens, vecs = rows * c.row_vecs;
  return vecs <= 32 * kKeep       ? launch_store<T, 1>(c, stream)
         : vecs <= 2 * 32 * kKeep ? launch_store<T, 2>(c, stream)
         : vecs <= 4 * 32 * kKeep ? launch_store<T, 4>(c, stream)
                                  : launch_store<T, 8>(c, stream);
}

template <typename T>
cudaError_t launch_load(const KvFp8Args &a, cudaStream_t stream) {
  constexpr uint32_t E = Row16<T>::kElems;
  LoadCall c;
  c.a = a;
  c.page_div = FastDiv(a.p.page_size);
  c.row_vecs = a.p.head_dim / E;
  c.row_div = FastDiv(c.row_vecs);
  c.vecs = c.row_vecs * a.p.n_kv_heads;
  c.wide = rows_wide(a, E);
  return launch_in_order(gdn_kv_load_kernel<T>, dim3((a.p.n_tokens + 3) / 4), 128, 0, stream, c);
}

}  // namespace

cudaError_t launch_kv_store_fp8(const KvFp8Args &a, cudaStream_t stream) {
  return a.p.dtype == GDN_DTYPE_BF16 ? launch_store<__nv_bfloat16>(a, stream) : launch_store<float>(a, stream);
}
cudaError_t launch_kv_load_fp8(const KvFp8Args &a, cudaStream_t stream) {
  return a.p.dtype == GDN_DTYPE_BF16 ? launch_load<__nv_bfloat16>(a, stream) : launch_load<float>(a, stream);
}

cudaError_t kv_fp8_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
