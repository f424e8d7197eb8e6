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
// takes a unit and keeps its rows in registers between the maximum and the codes;
// the heads of the same tokens go to neighbouring CTAs, so that rows which lie side
// by side are read at one time (23.1 -> 21.5 us for four prompts of 12 400 tokens
// together, 8 heads of 128, bf16).  The maximum is taken of the bits, two bf16 at a
// time, and values that are not finite are looked for only where it shows one.  With many tokens a team has
// up to a page of them, far apart and with no divisor in common with the page size: so each finds about one
// of a prompt's runs, and decodes, which are neighbours in the call, go to different teams.  (A team with
// neighbouring tokens took 100 decodes one after the other: with them and 100 prompts of up to 1000 tokens,
// 8 heads of 128, pages of 64, bf16, 55.9 -> 18.1 us; a run's length, which is then not among the slots
// already read, costs prompts alone 18.1 -> 19.4 us.  Reading a likely whole page's rows before its length
// is known: 22.1 us.)
//
// Measured on a GB300: those four prompts, pages of 64: 19.3 us, 4.0 TB/s, 0.59 of
// the copy bandwidth: instructions bound it (19 for an element at first: 24.9 us),
// and a team's life is a chain of slots, rows and codes with nothing of the next run
// on its way; pages of 16 and 128: 23.9 and 26.8 us; f32, pages of 16, 64 and 128: 53.6, 29.7
// and 54.0.  37 requests, decodes and two prompts of up to 333 tokens, f32, 2 heads of 256: 6.3 us.
// 64 decodes in pages of 16: 2.9 us, launch latency; 512 and 2048 decodes in pages of 16: 6.3 and
// 15.3 us, of 64: 13.7 and 46.5, of 128: 26.8 and 102 (0.4 and 1.8 for the bytes): a team has the
// warps that a whole page's rows need, of which a single token's use one row.
//
// Load.  A warp takes a token: 28 us for 33 000 tokens of 8 heads of 128 to bf16, 0.9
// of the copy bandwidth; to f32 45.8 us, 0.92.
#include <cuda_runtime.h>

#include <numeric>
#include <type_traits>

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
  static constexpr unsigned kInf = 0x7f800000u;
  // the largest magnitude, as bits, so far; of the finite ones only, with FINITE
  template <bool FINITE>
  __device__ __forceinline__ void raise(unsigned &m) const {
    const float f[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned b = __float_as_uint(f[i]) & 0x7fffffffu;
      m = max(m, FINITE && b >= kInf ? 0u : b);
    }
  }
  static __device__ __forceinline__ unsigned top(unsigned m) { return m; }  // as an f32's bits
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = x.x, f[1] = x.y, f[2] = x.z, f[3] = x.w; }
  __device__ __forceinline__ void put(const float (&f)[4]) { x = make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Row16<__nv_bfloat16> {
  static constexpr int kElems = 8;
  uint4 x;
  template <bool FINITE>
  __device__ __forceinline__ void raise(unsigned &m) const {
    const unsigned w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      unsigned b = w[i] & 0x7fff7fffu;
      if (FINITE) b &= ~__vcmpgeu2(b, 0x7f807f80u);
      m = __vmaxu2(m, b);
    }
  }
  static __device__ __forceinline__ unsigned top(unsigned m) { return max(m << 16, m & 0xffff0000u); }
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
  FastDiv page_div, rows_div;  // by the page size; by a token's rows of k and v
  FastDiv row_div;   // by the vectors of a row
  uint32_t at_once;  // rows that a team's threads take at once
  uint32_t window;   // tokens whose runs' beginnings a team looks for
  uint32_t windows;
  bool wide;         // rows of k and v are aligned to 16 bytes
};

template <typename T, int W>
__global__ void __launch_bounds__(W > 4 ? 32 * W : 128, W > 4 ? 4 : W > 2 ? 8 : 6) gdn_kv_store_kernel(const __grid_constant__ StoreCall c) {
  constexpr int E = Row16<T>::kElems, kTeams = W > 4 ? 1 : 4 / W;  // of a CTA
  __shared__ unsigned s_top[kTeams][W];
  const gdn_kv_fp8_params &p = c.a.p;
  const int lane = threadIdx.x & 31, team = threadIdx.x / (32 * W), me = threadIdx.x % (32 * W);
  auto meet = [&] {
    if constexpr (W == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;\n" ::"r"(1 + team), "n"(32 * W) : "memory");
  };
  // A thread keeps its place in a row, and goes through the rows of a run `at_once` apart.
  const int at_once = c.at_once, my_row = c.row_div.div(me), my_col = (me - my_row * static_cast<int>(c.row_div.d)) * E;
  const bool active = my_row < at_once;
  begin_in_order();
  // neighbouring CTAs have the heads of the same tokens, whose rows lie side by side
  const uint32_t group = c.rows_div.div(blockIdx.x), of = blockIdx.x - group * c.rows_div.d;
  const uint32_t unit = group * kTeams + team, which = of & 1, head = of >> 1;
  if (unit >= c.windows) return;  // the whole team
  const int n = static_cast<int>(p.n_tokens);
  const T *src = static_cast<const T *>(which ? c.a.v : c.a.k) + head * p.head_dim;
  const int64_t src_stride = which ? p.v_stride : p.k_stride;
  uint8_t *cache = static_cast<uint8_t *>(which ? c.a.v_cache : c.a.k_cache) + head * p.cache_head_stride;
  float *scales = (which ? c.a.v_scale : c.a.k_scale) + head;
  const int32_t *slots = c.a.slot_map;

  for (uint32_t base = 0; base < c.window; base += 32) {
    // The team's tokens lie `windows` apart, so that neighbouring decodes, a run each, go to different teams; the runs that begin
    // at them are the team's.
    const int64_t mine_at = unit + static_cast<int64_t>(base + lane) * c.windows;
    const bool have = base + lane < c.window && mine_at < n;
    const int i = have ? static_cast<int>(mine_at) : 0;
    const int slot_i = have ? slots[i] : -1, before = have && i ? slots[i - 1] : -1, next = have && i + 1 < n ? slots[i + 1] : -1;
    bool begins = false, more = false;
    if (slot_i >= 0) {
      const uint32_t page = c.page_div.div(slot_i);
      const bool same = before >= 0 && c.page_div.div(before) == page;
      begins = !(same && before == slot_i - 1);
      more = next - 1 == slot_i && c.page_div.div(next) == page;
      if (page >= p.n_pages) {
        if (begins) report(GDN_DEVICE_BAD_PAGE);
        begins = false;
      } else if (begins && same) {  // a page's tokens out of order
        report(GDN_DEVICE_BAD_REQUEST);
        begins = false;
      }
    }
    const unsigned longer = __ballot_sync(kFull, more);
    for (unsigned left = __ballot_sync(kFull, begins); left; left &= left - 1) {
      const int from = __ffs(left) - 1, first = __shfl_sync(kFull, i, from);
      const int slot = __shfl_sync(kFull, slot_i, from);
      const uint32_t page = c.page_div.div(slot);
      const int place = slot - static_cast<int>(page * p.page_size), most = static_cast<int>(p.page_size) - place;
      // tokens of the run: up to the first that does not follow
      int len = 1;
      for (bool go = longer >> from & 1; go;) {
        const int a = len + lane, b = a + 32;
        const bool on_a = a < most && a < n - first && slots[first + a] == slot + a;
        const bool on_b = b < most && b < n - first && slots[first + b] == slot + b;
        const unsigned e_a = __ballot_sync(kFull, !on_a), e_b = __ballot_sync(kFull, !on_b);
        len += e_a ? __ffs(e_a) - 1 : e_b ? __ffs(e_b) + 31 : 64;
        go = !e_a && !e_b;
      }
      float *scale_at = scales + static_cast<uint64_t>(page) * p.n_kv_heads;
      const float old = place ? *scale_at : 0.0f;
      uint8_t *rows = cache + page * p.cache_page_stride;
      const int mine = active ? len - my_row : 0;  // rows from this thread's first on
      const T *from_row = src + static_cast<int64_t>(first + my_row) * src_stride + my_col;
      const int64_t step = at_once * src_stride;
      // the largest magnitude: of all values, and where one of them is not finite, of the others
      Row16<T> keep[kKeep];
#pragma unroll
      for (int u = 0; u < kKeep; ++u)
        if (u * at_once < mine) keep[u] = load_row(from_row + u * step, c.wide);
      unsigned top_bits = 0;
      auto raise = [&](auto finite) {
        unsigned m = 0;
#pragma unroll
        for (int u = 0; u < kKeep; ++u)
          if (u * at_once < mine) keep[u].template raise<finite()>(m);
        for (int r = kKeep * at_once; r < mine; r += at_once) load_row(from_row + r / at_once * step, c.wide).template raise<finite()>(m);
        m = Row16<T>::top(m);
        m = __reduce_max_sync(kFull, m);
        if constexpr (W > 1) {
          if (lane == 0) s_top[team][me / 32] = m;
          meet();
#pragma unroll
          for (int w = 0; w < W; ++w) m = max(m, s_top[team][w]);
          meet();
        }
        top_bits = m;
      };
      raise(std::false_type{});
      const bool finite = top_bits < 0x7f800000u;
      if (!finite) raise(std::true_type{});
      const float top = __uint_as_float(top_bits);
      const float need = least_scale(top);
      const float scale = old > need && old <= 3.402823466e38f ? old : need, inv = 1.0f / scale;
      // the page's earlier tokens, on the new scale; those of a scale that is none (negative, infinite, NaN) are NaN
      if (place && scale != old) {
        const float by = old >= 0.0f && old <= 3.402823466e38f ? old * inv : __int_as_float(0x7fffffff);
        const int row16 = p.head_dim / 16, rows_at_once = 32 * W / row16, first_row = me / row16;
        for (int r = first_row < rows_at_once ? first_row : place; r < place; r += rows_at_once) {
          uint4 *q = reinterpret_cast<uint4 *>(rows + r * p.cache_slot_stride + me % row16 * 16);
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
      uint8_t *to_row = rows + static_cast<int64_t>(place + my_row) * p.cache_slot_stride + my_col;
      const int64_t to_step = at_once * p.cache_slot_stride;
      auto put = [&](const Row16<T> &v, uint8_t *to) {
        float f[E];
        v.get(f);
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] *= inv;
        if (!finite) {  // (a value that is not finite is not so after the product either)
#pragma unroll
          for (int e = 0; e < E; ++e) f[e] = fabsf(f[e]) <= 3.402823466e38f ? f[e] : __int_as_float(0x7fffffff);
        }
        if constexpr (E == 8)
          *reinterpret_cast<uint2 *>(to) = make_uint2(codes_of(f[0], f[1], f[2], f[3]), codes_of(f[4], f[5], f[6], f[7]));
        else
          *reinterpret_cast<unsigned *>(to) = codes_of(f[0], f[1], f[2], f[3]);
      };
#pragma unroll
      for (int u = 0; u < kKeep; ++u)
        if (u * at_once < mine) put(keep[u], to_row + u * to_step);
      for (int r = kKeep * at_once; r < mine; r += at_once) put(load_row(from_row + r / at_once * step, c.wide), to_row + r / at_once * to_step);
      meet();  // the old scale has been read
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
  const uint64_t units = static_cast<uint64_t>(p.n_tokens) * p.n_kv_heads * 2, enough = 152ull * 64 / W;
  c.window = static_cast<uint32_t>(units / enough);
  if (c.window < 1) c.window = 1;
  if (c.window > p.page_size) c.window = p.page_size;
  while (c.window < p.n_tokens && units / c.window > 1u << 30) c.window *= 2;  // CTAs are counted in 31 bits
  c.windows = (p.n_tokens + c.window - 1) / c.window;
  // a prompt's runs begin a page apart: with no divisor in common the teams get one each
  if (c.window > 1)
    while (std::gcd(c.windows, p.page_size) != 1) ++c.windows;
  c.rows_div = FastDiv(2 * p.n_kv_heads);
  c.at_once = 32 * W / c.row_div.d;
  return launch_in_order(gdn_kv_store_kernel<T, W>, dim3((c.windows + kTeams - 1) / kTeams * 2 * p.n_kv_heads), W > 4 ? 32 * W : 128, 0, stream, c);
}

template <typename T>
cudaError_t launch_store(const KvFp8Args &a, cudaStream_t stream) {
  constexpr uint32_t E = Row16<T>::kElems;
  StoreCall c;
  c.a = a;
  c.page_div = FastDiv(a.p.page_size);
  c.row_div = FastDiv(a.p.head_dim / E);
  c.wide = rows_wide(a, E);
  // warps enough for the longest run's rows to stay in registers (and for a row)
  const uint64_t rows = a.p.page_size < a.p.n_tokens ? a.p.page_size : a.p.n_tokens;
  auto holds = [&](uint64_t w) { return 32 * w / c.row_div.d * kKeep >= rows; };
  return holds(1)   ? launch_store<T, 1>(c, stream)
         : holds(2) ? launch_store<T, 2>(c, stream)
         : holds(4) ? launch_store<T, 4>(c, stream)
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
