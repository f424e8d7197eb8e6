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
// prompts and latency bounds decode steps.  A lane keeps one place in the head
// (E pairs, as two vectors: their halves, or neighbours) and goes through the
// rows of a token, a warp covering 32 / (places per head) rows at a time: the
// token's cosines stay in the lane's registers for all of them, several rows
// are on their way at once, and no warp waits for another.
//
// Measured on a GB300, back to back over three sets of buffers, as shares of the
// measured copy bandwidth (6783 GB/s): store of 16384 tokens, 32 + 2 x 8 heads of
// 128, bf16, three axes: 66 us, 0.91; gradient of 8209 tokens, 16 + 16 heads of 64:
// 15.2 us, 0.67 (short: a launch and the first loads are a third of it); 64 tokens:
// 3.1 us.  Cosines staged in shared memory for a CTA, one or several tokens a step,
// took 73 to 127 us for the first: a barrier per token, and fewer loads in flight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 2;  // rows a lane has on their way (1: 71, 3 with 5 CTAs: 71, 2: 70 us for 16384 tokens)
constexpr int kRowUnroll = 4;
constexpr int kCtasPerSm = 6;
constexpr uint32_t kEnoughWarps = 152 * kCtasPerSm * kWarps;  // what the GPU holds

// E contiguous elements, moved in one access of 16 bytes (or one element), and
// their values in f32; one rounding to nearest on the way back.
template <typename T, int E>
struct Vec;

template <int E>
struct alignas(4 * E) Vec<float, E> {
  float x[E];
  __device__ __forceinline__ void get(float (&f)[E]) const {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = x[e];
  }
  __device__ __forceinline__ void put(const float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = f[e];
  }
};

template <int E>
struct alignas(2 * E) Vec<__nv_bfloat16, E> {
  __nv_bfloat162 x[E / 2];
  __device__ __forceinline__ void get(float (&f)[E]) const {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float2 y = __bfloat1622float2(x[e]);
      f[2 * e] = y.x;
      f[2 * e + 1] = y.y;
    }
  }
  __device__ __forceinline__ void put(const float (&f)[E]) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) x[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  }
};

template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 x;
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __bfloat162float(x); }
  __device__ __forceinline__ void put(const float (&f)[1]) { x = __float2bfloat16_rn(f[0]); }
};

template <typename V>
__device__ __forceinline__ V from_lane(const V &v, int lane) {
  V y;
  const uint32_t *x = reinterpret_cast<const uint32_t *>(&v);
  uint32_t *to = reinterpret_cast<uint32_t *>(&y);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(V) / 4); ++i) to[i] = __shfl_sync(0xffffffffu, x[i], lane);
  return y;
}

// Rotates the E pairs of two vectors: (lo[e], hi[e]), or neighbours within lo, then hi.
template <typename T, int E>
__device__ __forceinline__ void rotate(Vec<T, E> &lo, Vec<T, E> &hi, const float (&c)[E], const float (&s)[E], bool inter) {
  float a[E], b[E];
  lo.get(a);
  hi.get(b);
  if (inter && E > 1) {
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const float x = a[2 * e], y = b[2 * e];
      a[2 * e] = x * c[e] - a[2 * e + 1] * s[e];
      a[2 * e + 1] = a[2 * e + 1] * c[e] + x * s[e];
      b[2 * e] = y * c[E / 2 + e] - b[2 * e + 1] * s[E / 2 + e];
      b[2 * e + 1] = b[2 * e + 1] * c[E / 2 + e] + y * s[E / 2 + e];
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = a[e];
      a[e] = x * c[e] - b[e] * s[e];
      b[e] = b[e] * c[e] + x * s[e];
    }
  }
  lo.put(a);
  hi.put(b);
}

constexpr uint32_t kMixed = 255;

struct RopeDivs {
  FastDiv parts, page;
  uint32_t n_parts;      // a token's rows are cut into this many parts, one per warp
  uint32_t part_rows;
  uint8_t place_axis[GDN_ROPE_MAX_DIM / 2];  // the axis of a place's E pairs; kMixed: several, or cos_sin only by the element
};

// Two vectors per lane: heads of 256 bytes or more, rotated in full as halves, and every layout that whole rows
// do not take.
template <typename T, int E>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) gdn_rope_kernel(const __grid_constant__ RopeArgs a,
                                                                        const RopeDivs dv) {
  using V = Vec<T, E>;
  const gdn_rope_params &p = a.p;
  const uint32_t half = p.rot_dim / 2, lane = threadIdx.x & 31;
  const bool store = a.v != nullptr, inter = (p.flags & GDN_ROPE_INTERLEAVED) != 0;
  const uint32_t places = p.head_dim / (2 * E), rot_places = p.rot_dim / (2 * E);
  // rows of a token: q heads, k heads, v heads
  const uint32_t k_row = p.n_q_heads, v_row = k_row + p.n_kv_heads;
  const uint32_t n_rows = store ? v_row + p.n_kv_heads : v_row;
  // the warp's rows at a time (one where a head has more places than the warp has lanes)
  const uint32_t at_once = places < 32 ? 32 / places : 1, my_row = places < 32 ? lane / places : 0;
  const bool active = my_row < at_once;
  begin_in_order();
  const uint32_t n_units = p.n_tokens * dv.n_parts;  // below 2^31: parts > 1 only with few tokens

  for (uint32_t j = places < 32 ? lane - my_row * places : lane; j < places; j += 32) {
    const bool turns = j < rot_places;
    // where q and k rows have this place's two vectors, and v rows
    // (halves of the rotated part, of the rest and of a v row, so that neighbouring lanes read neighbouring vectors)
    const uint32_t col = !turns ? p.rot_dim + (j - rot_places) * E : inter ? j * 2 * E : j * E;
    const uint32_t gap = !turns ? (p.head_dim - p.rot_dim) / 2 : inter ? E : half;
    const uint32_t v_col = j * E, v_gap = p.head_dim / 2;
    const uint32_t axis = turns ? dv.place_axis[j] : 0;

    const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit < n_units) {
      const uint32_t token = dv.parts.div(unit), part = unit - token * dv.n_parts;
      const uint32_t row1 = min(n_rows, (part + 1) * dv.part_rows);
      const int slot = store ? a.slot_map[token] : -1;
      const T *q = static_cast<const T *>(a.q) + token * p.q_stride, *k = static_cast<const T *>(a.k) + token * p.k_stride,
              *v = static_cast<const T *>(a.v) + token * p.v_stride;
      V lo[kUnroll], hi[kUnroll];
      auto load = [&](uint32_t r0) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const uint32_t r = r0 + my_row + u * at_once;
          if (r >= row1 || !active) continue;
          const T *src = r < k_row   ? q + r * p.head_dim + col
                         : r < v_row ? k + (r - k_row) * p.head_dim + col
                                     : v + (r - v_row) * p.head_dim + v_col;
          lo[u] = *reinterpret_cast<const V *>(src);
          hi[u] = *reinterpret_cast<const V *>(src + (r < v_row ? gap : v_gap));
        }
      };
      uint32_t r0 = part * dv.part_rows;
      load(r0);  // on its way while the cosines are looked up
      float c[E], s[E];
      if (turns) {
        if (E % 4 == 0 && axis != kMixed) {
          const int pos = a.positions[axis * p.positions_stride + token];
          if (static_cast<uint32_t>(pos) < p.n_positions) {
            const float *t = a.cos_sin + static_cast<uint64_t>(pos) * p.rot_dim + j * E;
#pragma unroll
            for (int e = 0; e + 3 < E; e += 4) {
              const float4 x = *reinterpret_cast<const float4 *>(t + e), y = *reinterpret_cast<const float4 *>(t + half + e);
              c[e] = x.x, c[e + 1] = x.y, c[e + 2] = x.z, c[e + 3] = x.w;
              s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
            }
          } else {  // no such row: the token's rotated values are NaN
#pragma unroll
            for (int e = 0; e < E; ++e) c[e] = s[e] = nanf("");
            report(GDN_DEVICE_BAD_POSITION);
          }
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const int pos = a.positions[p.axis_of_pair[j * E + e] * p.positions_stride + token];
            if (static_cast<uint32_t>(pos) < p.n_positions) {
              const float *t = a.cos_sin + static_cast<uint64_t>(pos) * p.rot_dim + j * E + e;
              c[e] = t[0];
              s[e] = t[half];
            } else {
              c[e] = s[e] = nanf("");
              report(GDN_DEVICE_BAD_POSITION);
            }
          }
        }
        if (p.flags & GDN_ROPE_INVERSE) {
#pragma unroll
          for (int e = 0; e < E; ++e) s[e] = -s[e];
        }
      }
      long long slot_at = -1;  // element offset of the token's slot in the caches; -1: k and v go nowhere
      if (slot >= 0) {
        const uint32_t page = dv.page.div(static_cast<uint32_t>(slot));
        if (page < p.n_pages)
          slot_at = page * p.cache_page_stride + static_cast<int64_t>(slot - page * p.page_size) * p.cache_slot_stride;
        else
          report(GDN_DEVICE_BAD_PAGE);
      }
      while (r0 < row1) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const uint32_t r = r0 + my_row + u * at_once;
          if (r >= row1 || !active) continue;
          if (turns && r < v_row) rotate<T, E>(lo[u], hi[u], c, s, inter);
          T *dst;
          if (r < k_row) {
            dst = static_cast<T *>(a.q_out) + token * p.q_out_stride + r * p.head_dim + col;
          } else if (!store) {
            dst = static_cast<T *>(a.k_out) + token * p.k_out_stride + (r - k_row) * p.head_dim + col;
          } else {
            if (slot_at < 0) continue;
            dst = r < v_row ? static_cast<T *>(a.k_cache) + slot_at + (r - k_row) * p.cache_head_stride + col
                            : static_cast<T *>(a.v_cache) + slot_at + (r - v_row) * p.cache_head_stride + v_col;
          }
          *reinterpret_cast<V *>(dst) = lo[u];
          *reinterpret_cast<V *>(dst + (r < v_row ? gap : v_gap)) = hi[u];
        }
        r0 += kUnroll * at_once;
        load(r0);
      }
    }
  }
}

// Whole rows: a lane takes one vector, and a warp reads its rows as they lie.
// Where the two vectors of a pair would be pieces of 64 bytes or less of two
// accesses -- short rows, partial rotation, interleaved pairs, whose pieces
// alternate -- the cache's tags, not its bytes, would bound the form above
// (gradient of 8209 tokens of 16 + 16 heads of 64, bf16: 20.2 us there, 15.2
// here; store of 2630 tokens, 32 + 2 x 4 heads of 128, interleaved: 28.6 and
// 15.3).  A half's other half comes from the lane that has it.
template <typename T, int E, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) gdn_rope_rows_kernel(const __grid_constant__ RopeArgs a,
                                                                             const RopeDivs dv) {
  using V = Vec<T, E>;
  constexpr int kPairs = INTER ? E / 2 : E;  // whose cosines a lane needs
  const gdn_rope_params &p = a.p;
  const uint32_t half = p.rot_dim / 2, lane = threadIdx.x & 31;
  const bool store = a.v != nullptr, inverse = (p.flags & GDN_ROPE_INVERSE) != 0;
  const uint32_t k_row = p.n_q_heads, v_row = k_row + p.n_kv_heads;
  const uint32_t n_rows = store ? v_row + p.n_kv_heads : v_row;
  // rows at a time; this lane's vector of its row
  const uint32_t places = p.head_dim / E, at_once = 32 / places, my_row = lane / places, j = lane - my_row * places;
  const bool active = my_row < at_once;
  const uint32_t rot_half = half / E;  // vectors of a rotated half
  const bool turns = j < 2 * rot_half, second = j >= rot_half;
  const uint32_t pair0 = INTER ? j * kPairs : (second ? j - rot_half : j) * E;
  const uint32_t other = !INTER && turns ? (second ? lane - rot_half : lane + rot_half) : lane;
  begin_in_order();
  const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (unit >= p.n_tokens * dv.n_parts) return;  // the whole warp
  const uint32_t token = dv.parts.div(unit), part = unit - token * dv.n_parts;
  const uint32_t row1 = min(n_rows, (part + 1) * dv.part_rows);
  const int slot = store ? a.slot_map[token] : -1;
  const T *q = static_cast<const T *>(a.q) + token * p.q_stride + j * E,
          *k = static_cast<const T *>(a.k) + token * p.k_stride + j * E,
          *v = static_cast<const T *>(a.v) + (store ? token * p.v_stride + j * E : 0);
  V x[kRowUnroll];
  auto load = [&](uint32_t r0) {
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const uint32_t r = r0 + my_row + u * at_once;
      if (r >= row1 || !active) continue;
      x[u] = *reinterpret_cast<const V *>(r < k_row   ? q + r * p.head_dim
                                          : r < v_row ? k + (r - k_row) * p.head_dim
                                                      : v + (r - v_row) * p.head_dim);
    }
  };
  uint32_t r0 = part * dv.part_rows;
  load(r0);  // on its way while the cosines are looked up
  float c[kPairs], s[kPairs];
  if (turns && active) {
    const uint32_t axis = dv.place_axis[j];
    if (kPairs % 4 == 0 && axis != kMixed) {
      const int pos = a.positions[axis * p.positions_stride + token];
      if (static_cast<uint32_t>(pos) < p.n_positions) {
        const float *t = a.cos_sin + static_cast<uint64_t>(pos) * p.rot_dim + pair0;
#pragma unroll
        for (int e = 0; e + 3 < kPairs; e += 4) {
          const float4 y = *reinterpret_cast<const float4 *>(t + e), z = *reinterpret_cast<const float4 *>(t + half + e);
          c[e] = y.x, c[e + 1] = y.y, c[e + 2] = y.z, c[e + 3] = y.w;
          s[e] = z.x, s[e + 1] = z.y, s[e + 2] = z.z, s[e + 3] = z.w;
        }
      } else {  // no such row: the token's rotated values are NaN
#pragma unroll
        for (int e = 0; e < kPairs; ++e) c[e] = s[e] = nanf("");
        report(GDN_DEVICE_BAD_POSITION);
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        const int pos = a.positions[p.axis_of_pair[pair0 + e] * p.positions_stride + token];
        if (static_cast<uint32_t>(pos) < p.n_positions) {
          const float *t = a.cos_sin + static_cast<uint64_t>(pos) * p.rot_dim + pair0 + e;
          c[e] = t[0];
          s[e] = t[half];
        } else {
          c[e] = s[e] = nanf("");
          report(GDN_DEVICE_BAD_POSITION);
        }
      }
    }
    // of halves, a pair's first element takes -s times the other, its second s
    if (inverse != (!INTER && !second)) {
#pragma unroll
      for (int e = 0; e < kPairs; ++e) s[e] = -s[e];
    }
  }
  long long slot_at = -1;  // element offset of the token's slot in the caches; -1: k and v go nowhere
  if (slot >= 0) {
    const uint32_t page = dv.page.div(static_cast<uint32_t>(slot));
    if (page < p.n_pages)
      slot_at = page * p.cache_page_stride + static_cast<int64_t>(slot - page * p.page_size) * p.cache_slot_stride;
    else
      report(GDN_DEVICE_BAD_PAGE);
  }
  while (r0 < row1) {
#pragma unroll
    for (int u = 0; u < kRowUnroll; ++u) {
      const uint32_t r = r0 + my_row + u * at_once;
      V y;
      if constexpr (!INTER) y = from_lane(x[u], other);  // every lane takes part
      if (r >= row1 || !active) continue;
      if (turns && r < v_row) {
        float mine[E];
        x[u].get(mine);
        if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < kPairs; ++e) {
            const float f = mine[2 * e], g = mine[2 * e + 1];
            mine[2 * e] = f * c[e] - g * s[e];
            mine[2 * e + 1] = g * c[e] + f * s[e];
          }
        } else {
          float theirs[E];
          y.get(theirs);
#pragma unroll
          for (int e = 0; e < E; ++e) mine[e] = mine[e] * c[e] + theirs[e] * s[e];
        }
        x[u].put(mine);
      }
      T *dst;
      if (r < k_row) {
        dst = static_cast<T *>(a.q_out) + token * p.q_out_stride + r * p.head_dim;
      } else if (!store) {
        dst = static_cast<T *>(a.k_out) + token * p.k_out_stride + (r - k_row) * p.head_dim;
      } else {
        if (slot_at < 0) continue;
        dst = r < v_row ? static_cast<T *>(a.k_cache) + slot_at + (r - k_row) * p.cache_head_stride
                        : static_cast<T *>(a.v_cache) + slot_at + (r - v_row) * p.cache_head_stride;
      }
      *reinterpret_cast<V *>(dst + j * E) = x[u];
    }
    r0 += kRowUnroll * at_once;
    load(r0);
  }
}

// places: what a row is cut into among lanes; n: neighbouring pairs of one place, the axis of `marked` places asked for.
RopeDivs divide_up(const RopeArgs &a, uint32_t places, uint32_t marked, uint32_t n) {
  const gdn_rope_params &p = a.p;
  const uint32_t at_once = places < 32 ? 32 / places : 1;
  const uint32_t rows = p.n_q_heads + p.n_kv_heads * (a.v ? 2 : 1);
  RopeDivs dv;
  dv.page = FastDiv(p.page_size ? p.page_size : 1);
  // A token's rows to one warp, so that its cosines are read once; with fewer
  // tokens to several warps, down to one step of rows each: latency.
  const uint32_t steps = (rows + at_once - 1) / at_once;
  uint32_t parts = p.n_tokens < kEnoughWarps ? kEnoughWarps / p.n_tokens : 1;
  if (parts > steps) parts = steps;
  dv.part_rows = (steps + parts - 1) / parts * at_once;
  dv.n_parts = (rows + dv.part_rows - 1) / dv.part_rows;
  dv.parts = FastDiv(dv.n_parts);
  const bool wide = n % 4 == 0 && reinterpret_cast<uintptr_t>(a.cos_sin) % 16 == 0 && p.rot_dim % 8 == 0;
  for (uint32_t j = 0; j < marked; ++j) {
    const uint8_t *x = p.axis_of_pair + j * n % (p.rot_dim / 2);  // a second half's places have the first's pairs
    bool one = wide && x[0] < kMixed;
    for (uint32_t e = 1; e < n; ++e) one = one && x[e] == x[0];
    dv.place_axis[j] = one ? x[0] : kMixed;
  }
  return dv;
}

uint32_t ctas_of(const RopeArgs &a, const RopeDivs &dv) {
  return static_cast<uint32_t>((static_cast<uint64_t>(a.p.n_tokens) * dv.n_parts + kWarps - 1) / kWarps);
}

template <typename T, int E>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  const RopeDivs dv = divide_up(a, a.p.head_dim / (2 * E), a.p.rot_dim / (2 * E), E);
  return launch_in_order(gdn_rope_kernel<T, E>, dim3(ctas_of(a, dv)), kThreads, 0, stream, a, dv);
}

template <typename T, int E>
cudaError_t launch_vectors(const RopeArgs &a, cudaStream_t stream) {
  const gdn_rope_params &p = a.p;
  const bool inter = (p.flags & GDN_ROPE_INTERLEAVED) != 0;
  if (p.head_dim / E > 32 || !(inter || p.rot_dim < p.head_dim || p.head_dim * sizeof(T) <= 128)) return launch<T, E>(a, stream);
  const RopeDivs dv = divide_up(a, p.head_dim / E, p.rot_dim / E, inter ? E / 2 : E);
  return inter ? launch_in_order(gdn_rope_rows_kernel<T, E, true>, dim3(ctas_of(a, dv)), kThreads, 0, stream, a, dv)
               : launch_in_order(gdn_rope_rows_kernel<T, E, false>, dim3(ctas_of(a, dv)), kThreads, 0, stream, a, dv);
}

// Whether every access of E elements is aligned and none crosses the rotated
// part's or a head's end.
bool vectors_fit(const RopeArgs &a, uint32_t e, uint32_t elem) {
  const gdn_rope_params &p = a.p;
  if (p.head_dim % (2 * e) || p.rot_dim % (2 * e)) return false;
  const void *ptrs[] = {a.q, a.k, a.v, a.q_out, a.k_out, a.k_cache, a.v_cache};
  for (const void *x : ptrs)
    if (reinterpret_cast<uintptr_t>(x) % (e * elem)) return false;
  const int64_t strides[] = {p.q_stride, p.k_stride, a.v ? p.v_stride : 0, p.q_out_stride,
                             a.k_out ? p.k_out_stride : 0, a.v ? p.cache_page_stride : 0,
                             a.v ? p.cache_head_stride : 0, a.v ? p.cache_slot_stride : 0};
  for (int64_t s : strides)
    if (s % e) return false;
  return true;
}

// 16-byte vectors where they fit, 8-byte ones for heads such as 72 bf16
// elements, single elements for any other layout.
template <typename T>
cudaError_t launch_type(const RopeArgs &a, cudaStream_t stream) {
  constexpr int E = 16 / sizeof(T);
  return vectors_fit(a, E, sizeof(T))       ? launch_vectors<T, E>(a, stream)
         : vectors_fit(a, E / 2, sizeof(T)) ? launch_vectors<T, E / 2>(a, stream)
                                            : launch<T, 1>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  return a.p.dtype == GDN_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<float>(a, stream);
}

cudaError_t rope_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
