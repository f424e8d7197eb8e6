// What the attention kernels over a paged cache share (attn_paged.cu, attn_fp8.cu):
// the call as the kernels see it, how its work is split over the CTAs, and the
// join of an item's parts.
//
// The work of a call is a list of units: 64 keys, and kItemUnits, which the file
// that includes this one defines, for an item's begin and end (an item is a request's key head and block of rows).  The lengths
// are on the device, so every CTA takes the prefix sum of the requests' units and
// then the same share of the whole list.  A share may begin and end inside an item:
// such ends leave unnormalised sums with their running maximum in the workspace
// (at most two per CTA), and a second launch joins them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "device_io.cuh"
#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr int kSub = 16;   // keys of a matrix tile
constexpr int kUnit = 64;  // keys per unit of work
constexpr int kMostTile = 32;  // largest tile of a key group
constexpr int kSms = 152;
constexpr int kJoinWarps = 8;

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;  // the lowest finite f32

__device__ __forceinline__ unsigned smem_u32(const void *p) {
  return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ unsigned movmatrix_trans(unsigned x) {
  unsigned y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void cp_async_16_or_zero(unsigned smem, const void *gmem, bool read) {
  const int n = read ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "r"(n) : "memory");
}

// ------------------------------------------------------------ the call, as the kernels see it

// An item that begins in one CTA and goes on in later ones: what the join needs to know of it.
struct alignas(16) Split {
  int slot;      // of its first part; -1: no item is split here
  int last;      // the last CTA that has a part of it
  int row0, rows;  // its first row, and the rows of its key head: row = token * group + query head
  int t0;        // the request's first row of q
  int head0;     // its key head's first query head
  int before;    // keys that are before the request's window of tokens; below 0, its first tokens see none
};

struct Call {
  const void *q, *k, *v;
  const float *k_scale, *v_scale;  // of an 8-bit cache: [page][key head]
  const int32_t *table, *kv_lens, *token_start;
  void *out;
  float *part;     // [2 * ctas][rows][D] unnormalised sums
  float2 *part_ml; // [2 * ctas][rows] running maximum (log2 domain) and sum
  Split *splits;   // [ctas] the split item that begins in the CTA
  uint32_t n_seqs, n_tokens, n_kv, group, max_pages, page_size, n_pages, window;
  float scale_log2;
  int64_t q_stride, out_stride, page_stride, head_stride, slot_stride;
  FastDiv page_div, group_div;
  bool whole_tiles;  // pages hold whole tiles
  bool whole_items;  // no item is split
  bool out_wide;     // output rows are aligned to four elements
  // of an 8-bit cache's call:
  bool q_wide;       // rows of q are aligned to 16 bytes
  uint32_t box;      // rows of a box of tensor copies
  uint32_t wait_clocks;  // after which a wait runs out
};

// A request's share of the work.
struct Request {
  int t0, tokens;   // its rows of q
  int len, first;   // its keys: those that at least one token sees lie in [first, len)
  int blocks;       // row blocks per key head
  int tiles;        // units of keys per (key head, row block); 1 when there is no key
  bool bad;
  // where its units begin; tiles begin at multiples of their size
  __device__ __forceinline__ int lo() const { return first & ~(kMostTile - 1); }
  __device__ __forceinline__ long long units(const Call &c) const {
    return tokens > 0 ? static_cast<long long>(c.n_kv) * blocks * (tiles + kItemUnits) : 0;
  }
};

template <int ROWS>
__device__ __forceinline__ Request request(const Call &c, uint32_t s) {
  Request r;
  r.bad = false;
  int t0 = s, t1 = s + 1;
  if (c.token_start) {
    t0 = c.token_start[s];
    t1 = c.token_start[s + 1];
  }
  const int n = static_cast<int>(c.n_tokens);
  if (t0 < 0 || t1 < t0 || t1 > n) {  // rows that q does not have are left out
    r.bad = true;
    t0 = min(max(t0, 0), n);
    t1 = min(max(t1, t0), n);
  }
  r.t0 = t0;
  r.tokens = t1 - t0;
  int len = c.kv_lens[s];
  const long long most = static_cast<long long>(c.max_pages) * c.page_size;
  if (len < 0 || len > most) {
    r.bad = true;
    len = len < 0 ? 0 : static_cast<int>(most);
  }
  r.len = len;
  const long long lo = c.window ? static_cast<long long>(len) - r.tokens + 1 - c.window : 0;
  r.first = static_cast<int>(lo > 0 ? (lo < len ? lo : len) : 0);
  const long long rows = static_cast<long long>(r.tokens) * c.group;
  r.blocks = static_cast<int>((rows + ROWS - 1) / ROWS);
  const int tiles = (len - r.lo() + kUnit - 1) / kUnit;
  r.tiles = tiles > 0 ? tiles : 1;
  return r;
}

// a / b for a >= 0, in 32 bits where they hold a (64-bit division is a long subroutine).
__device__ __forceinline__ long long divide(long long a, uint32_t b) {
  return a >> 32 ? a / b : static_cast<uint32_t>(a) / b;
}
// x - window, no lower than any key index needs.
__device__ __forceinline__ int less_window(int x, uint32_t window) {
  const long long y = static_cast<long long>(x) - window;
  return y < -(1 << 30) ? -(1 << 30) : static_cast<int>(y);
}
// CTA x of `ctas` takes units [start(x), start(x + 1)).
__device__ __forceinline__ long long share_start(long long total, int ctas, int x) {
  return divide(total * x, ctas);
}

// Four neighbouring results, rounded once; in one store where rows are aligned to it.
__device__ __forceinline__ void put4(float *o, const float (&x)[4], bool wide) {
  if (wide) {
    *reinterpret_cast<float4 *>(o) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = x[e];
  }
}
__device__ __forceinline__ void put4(__nv_bfloat16 *o, const float (&x)[4], bool wide) {
  if (wide) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2 *>(o) = make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = __float2bfloat16_rn(x[e]);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// One (request, key head, row block) item of a CTA's share, or the part of it
// that lies in the share.
template <int ROWS, int KW, int TILE>
struct Item {
  uint32_t seq;
  Request r;
  long long in_seq;      // units of the request before the share's next one
  int item;              // head * r.blocks + block
  int units;             // of the item in this share
  int tile0, tile1;      // its units of keys
  int k0, k1;            // its keys

  // The next part of the share: [u, u1) are the share's units still to come, the first of them unit in_seq of
  // request seq.  An item's first kItemUnits units hold no keys.
  __device__ __forceinline__ bool find(const Call &c, long long &u, long long u1) {
    while (u < u1) {
      while (in_seq >= r.units(c)) {
        in_seq = 0;
        if (++seq >= c.n_seqs) return false;
        r = request<ROWS>(c, seq);
      }
      const int all = r.tiles + kItemUnits;
      item = static_cast<int>(divide(in_seq, all));
      const int at = static_cast<int>(in_seq - static_cast<long long>(item) * all);
      units = static_cast<int>(min(static_cast<long long>(all - at), u1 - u));
      if (c.whole_items) {  // to the share that has its first unit
        if (at > 0) {
          pass(u);
          continue;
        }
        units = all;
      }
      tile0 = max(0, at - kItemUnits);
      tile1 = at + units - kItemUnits;
      if (tile1 > tile0) {
        k0 = r.lo() + tile0 * kUnit;
        k1 = min(r.len, r.lo() + tile1 * kUnit);
        return true;
      }
      pass(u);
    }
    return false;
  }
  __device__ __forceinline__ void pass(long long &u) {
    u += units;
    in_seq += units;
  }
  // Tiles of this part that key group `kg` takes: k0 + TILE (kg + KW i).
  __device__ __forceinline__ int tiles_of(int kg) const {
    const int first = k0 + TILE * kg;
    return first < k1 ? (k1 - first + TILE * KW - 1) / (TILE * KW) : 0;
  }
};

// A CTA's share of the units: [u0, u1) of `total`.
struct Share {
  int cta, ctas;  // nothing to do where cta >= ctas
  long long total, u0, u1;
};

// The share of this CTA, by the prefix sum of the requests' units, a contiguous run of requests per thread.  `seq` and
// `offset` become the request of its first unit and the unit's place in the request, `first` that request.  Every thread
// of the CTA takes part.
template <int ROWS, int WARPS>
__device__ __forceinline__ Share take_share(const Call &c, long long (&scan)[WARPS], uint32_t &seq, long long &offset,
                                            Request *first = nullptr) {
  constexpr int kThreads = 32 * WARPS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t per = (c.n_seqs + kThreads - 1) / kThreads;
  const uint32_t s_first = min(tid * per, c.n_seqs), s_last = min(s_first + per, c.n_seqs);
  long long mine = 0;
  bool bad = false;
  for (uint32_t s = s_first; s < s_last; ++s) {
    const Request r = request<ROWS>(c, s);
    mine += r.units(c);
    bad |= r.bad;
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += scan[w];
    total += scan[w];
  }
  before += inc - mine;
  if (bad && blockIdx.x == 0) report(GDN_DEVICE_BAD_REQUEST);
  Share sh;
  sh.total = total;
  sh.ctas = static_cast<int>(min(total, static_cast<long long>(gridDim.x)));
  sh.cta = blockIdx.x;
  if (tid == 0) c.splits[sh.cta].slot = -1;
  sh.u0 = sh.u1 = 0;
  if (sh.cta >= sh.ctas) return sh;
  sh.u0 = share_start(total, sh.ctas, sh.cta);
  sh.u1 = share_start(total, sh.ctas, sh.cta + 1);
  if (sh.u0 >= before && sh.u0 < before + mine) {
    long long at = before;
    for (uint32_t s = s_first; s < s_last; ++s) {
      const Request r = request<ROWS>(c, s);
      const long long n = r.units(c);
      if (sh.u0 < at + n) {
        if (first) *first = r;
        seq = s;
        offset = sh.u0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  return sh;
}

// ------------------------------------------------------------ the join

// The item that begins in main CTA blockIdx.x and goes on in later ones: CTA (x, y)
// joins its rows y * PER .. + PER, each by 8 / PER warps that take its parts in
// turn, a part by D / 4 lanes.
template <typename T, int D, int ROWS, int PER>
__global__ void __launch_bounds__(32 * kJoinWarps) gdn_attn_join_kernel(const __grid_constant__ Call c) {
  constexpr int kLanes = D / 4 < 32 ? D / 4 : 32, kVecs = D / 4 / kLanes;
  constexpr int kTeams = kJoinWarps * (32 / kLanes), kTeam = kTeams / PER;  // groups of lanes: in all, of a row
  constexpr int kAhead = 8;                                                 // parts a group has on their way
  __shared__ float4 s_acc[kTeams][D / 4];
  __shared__ float s_m[kTeams], s_den[kTeams];
  begin_in_order();
  const Split sp = c.splits[blockIdx.x];
  if (sp.slot < 0) return;
  const int team = threadIdx.x / kLanes, lane = threadIdx.x % kLanes, mine = team / kTeam, member = team % kTeam;
  const int row = blockIdx.y * PER + mine, item_row = sp.row0 + row;
  const int x0 = blockIdx.x, n = sp.last - x0 + 1;
  float4 acc[kVecs] = {};
  float m = kLowest, den = 0.0f;
  for (int i0 = member; i0 < n; i0 += kTeam * kAhead) {
    float2 ml[kAhead];
    float4 y[kAhead][kVecs];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const int i = i0 + a * kTeam;
      if (i < n && item_row < sp.rows) {
        const size_t at = static_cast<size_t>(i == 0 ? sp.slot : 2 * (x0 + i)) * ROWS + row;
        ml[a] = c.part_ml[at];
#pragma unroll
        for (int j = 0; j < kVecs; ++j) y[a][j] = *(reinterpret_cast<const float4 *>(c.part + at * D) + j * kLanes + lane);
      } else {
        ml[a] = make_float2(kLowest, 0.0f);
#pragma unroll
        for (int j = 0; j < kVecs; ++j) y[a][j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      const float top = fmaxf(m, ml[a].x), f = exp2_fast(ml[a].x - top), g = exp2_fast(m - top);
      den = den * g + f * ml[a].y;
#pragma unroll
      for (int j = 0; j < kVecs; ++j) {
        acc[j].x = acc[j].x * g + f * y[a][j].x;
        acc[j].y = acc[j].y * g + f * y[a][j].y;
        acc[j].z = acc[j].z * g + f * y[a][j].z;
        acc[j].w = acc[j].w * g + f * y[a][j].w;
      }
      m = top;
    }
  }
#pragma unroll
  for (int j = 0; j < kVecs; ++j) s_acc[team][j * kLanes + lane] = acc[j];
  if (lane == 0) {
    s_m[team] = m;
    s_den[team] = den;
  }
  __syncthreads();
  if (item_row >= sp.rows) return;
  float top = kLowest;
#pragma unroll
  for (int w = 0; w < kTeam; ++w) top = fmaxf(top, s_m[mine * kTeam + w]);
  den = 0.0f;
#pragma unroll
  for (int w = 0; w < kTeam; ++w) den += exp2_fast(s_m[mine * kTeam + w] - top) * s_den[mine * kTeam + w];
  const int t = c.group_div.div(item_row);
  T *o = static_cast<T *>(c.out) + static_cast<int64_t>(sp.t0 + t) * c.out_stride +
         static_cast<int64_t>(sp.head0 + (item_row - t * static_cast<int>(c.group))) * D;
  const bool empty = sp.before + t < 0 && !isnan(den);
  for (int d = member * kLanes + lane; d < D; d += kLanes * kTeam) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kTeam; ++w)
      sum += exp2_fast(s_m[mine * kTeam + w] - top) * reinterpret_cast<const float *>(s_acc[mine * kTeam + w])[d];
    Act<T>::put(o + d, empty ? 0.0f : sum / den);
  }
}

// ------------------------------------------------------------ host

// Rows that a request's newest tokens take per key head, on average: what the
// shape of a call is chosen by (longer windows take several row blocks).
inline uint64_t rows_of(const gdn_attn_params &p) {
  const uint64_t window = (p.n_tokens + static_cast<uint64_t>(p.n_seqs) - 1) / p.n_seqs;
  return window * (p.n_q_heads / p.n_kv_heads);
}

// The call but for what a kernel's shape decides.
inline Call call_of(const gdn_attn_params &p, const void *q, const void *k, const void *v, const int32_t *table,
                    const int32_t *kv_lens, const int32_t *token_start, void *out) {
  Call c = {};
  c.q = q;
  c.k = k;
  c.v = v;
  c.table = table;
  c.kv_lens = kv_lens;
  c.token_start = token_start;
  c.out = out;
  c.n_seqs = p.n_seqs;
  c.n_tokens = p.n_tokens;
  c.n_kv = p.n_kv_heads;
  c.group = p.n_q_heads / p.n_kv_heads;
  c.max_pages = p.max_pages;
  c.page_size = p.page_size;
  c.n_pages = p.n_pages;
  c.window = p.window;
  c.scale_log2 = p.scale * kLog2e;
  c.q_stride = p.q_stride;
  c.out_stride = p.out_stride;
  c.page_stride = p.cache_page_stride;
  c.head_stride = p.cache_head_stride;
  c.slot_stride = p.cache_slot_stride;
  c.page_div = FastDiv(p.page_size);
  c.group_div = FastDiv(c.group);
  const uintptr_t four = p.dtype == GDN_DTYPE_BF16 ? 8 : 16;
  c.out_wide = reinterpret_cast<uintptr_t>(out) % four == 0 && p.out_stride % 4 == 0;
  return c;
}

// Few items have many parts each: several warps per row; many have few: a warp per row.
template <typename T, int D, int ROWS>
cudaError_t launch_join(const Call &c, int ctas, bool few, cudaStream_t stream) {
  constexpr int kFewPer = ROWS / 4 < kJoinWarps ? ROWS / 4 : kJoinWarps;
  return launch_in_order(few ? gdn_attn_join_kernel<T, D, ROWS, kFewPer> : gdn_attn_join_kernel<T, D, ROWS, kJoinWarps>,
                         dim3(ctas, ROWS / (few ? kFewPer : kJoinWarps)), 32 * kJoinWarps, 0, stream, c);
}

inline size_t part_floats(int ctas, int rows, int d) { return static_cast<size_t>(2) * ctas * rows * d; }

}  // namespace
}  // namespace gdn
