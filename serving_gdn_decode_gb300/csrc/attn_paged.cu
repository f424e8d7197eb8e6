// Attention of each request's newest tokens over its paged key-value cache
// (gdn_attn_paged): out = sum_j softmax_j(scale q.k_j) v_j over the keys a
// token sees, for windows of one token (decode) to a few (verification).
//
// What bounds it.  Every cached key and value is read once and used for
// group x window rows, 2 to about 100 flops a byte in bf16: HBM bounds it, far
// from the tensor cores' rate, so the kernel is built around keeping loads in
// flight.  A token's rows sit on the N side of the matrix instruction (S^T = K
// Q^T, O^T = V^T P^T): N is 8 there, so a group of 1 to 8 query heads wastes
// the least, and accumulators stay small enough for registers.  The warp-level
// mma.sync serves this (about a tenth of its rate is needed); a tcgen05 tile
// would put 128 keys on the M side for the same 8 columns and pay tensor-memory
// round trips between two tiny products.
//
// Split over the length.  The work of a call is a list of units of 64 keys,
// ordered by (request, key head, row block, keys); the lengths are on the
// device, so every CTA takes the prefix sum of the requests' units and then the
// same share of the whole list, whatever the lengths are.  A CTA's share may
// begin and end inside an (request, head, row block) item: such ends leave
// unnormalised sums with their running maximum in the workspace (at most two
// per CTA), and a second launch joins them; an item that lies in one CTA goes
// straight to the output.  No atomics: the order of every sum is fixed by the
// sizes.
//
// Inside a CTA each of the 4 warps takes every fourth 16-key tile of the item
// with a softmax state of its own, and the four are joined at the item's end;
// so the main loop has no barrier between warps.  Each warp feeds itself
// through a ring of half tiles (16 rows of K, then the same rows of V) with
// 16-byte asynchronous copies, which follow any page size, stride and tile
// edge; rows past the end arrive as zeros, so stale values of a page never meet
// the products.
//
// Precision.  f32: each operand is split in two TF32 halves and three products
// are taken, so products and sums are good to f32.  bf16: K, V and q are exact
// in the products; the probabilities are split in two bf16 halves (two products
// instead of one), which keeps the result at f32 quality until its one rounding
// at the end.  The maximum, the sum and all accumulators are f32.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_io.cuh"
#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16;               // keys per warp tile
constexpr int kUnit = kTile * kWarps;   // keys per unit of work
constexpr int kSms = 152;
constexpr int kJoinWarps = 4;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------ matrix instructions

__device__ __forceinline__ unsigned smem_u32(const void *p) {
  return static_cast<unsigned>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void ldmatrix_x4(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(unsigned (&r)[4], unsigned addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ unsigned movmatrix_trans(unsigned x) {
  unsigned y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// c += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a (16 x 8) b (8 x 8), TF32
__device__ __forceinline__ void mma_tf32(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ unsigned to_tf32(float x) {
  unsigned y;
  asm("cvt.rna.tf32.f32 %0, %1;\n" : "=r"(y) : "f"(x));
  return y;
}
// x = hi + lo up to 2^-22 |x|, both TF32, rounded to nearest.
struct Tf32Pair {
  unsigned hi, lo;
  __device__ __forceinline__ explicit Tf32Pair(float x) {
    hi = to_tf32(x);
    lo = to_tf32(x - __uint_as_float(hi));
  }
};

__device__ __forceinline__ void cp_async_16_or_zero(unsigned smem, const void *gmem, bool read) {
  const int n = read ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(smem), "l"(gmem), "r"(n) : "memory");
}

// ------------------------------------------------------------ the call, as the kernels see it

struct Call {
  const void *q, *k, *v;
  const int32_t *table, *kv_lens, *token_start;
  void *out;
  float *part;     // [2 * ctas][rows][D] unnormalised sums
  float2 *part_ml; // [2 * ctas][rows] running maximum (log2 domain) and sum
  int4 *meta;      // [ctas] the split item that begins in the CTA: request, head and row block, last CTA, slot of its part (-1: none)
  uint32_t n_seqs, n_tokens, n_kv, group, max_pages, page_size, n_pages, window;
  float scale_log2;
  int64_t q_stride, out_stride, page_stride, head_stride, slot_stride;
  FastDiv page_div, group_div;
};

// A request's share of the work.
struct Request {
  int t0, tokens;   // its rows of q
  int len, lo;      // its keys: [lo, len) are seen by at least one token
  int blocks;       // row blocks per key head
  int tiles;        // units per (key head, row block); 1 when there is no key
  bool bad;
  __device__ __forceinline__ long long units(const Call &c) const {
    return tokens > 0 ? static_cast<long long>(c.n_kv) * blocks * tiles : 0;
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
  r.lo = static_cast<int>(lo > 0 ? (lo < len ? lo : len) : 0);
  const long long rows = static_cast<long long>(r.tokens) * c.group;
  r.blocks = static_cast<int>((rows + ROWS - 1) / ROWS);
  const int tiles = (len - r.lo + kUnit - 1) / kUnit;
  r.tiles = tiles > 0 ? tiles : 1;
  return r;
}

// CTA x of `ctas` takes units [start(x), start(x + 1)).
__device__ __forceinline__ long long share_start(long long total, int ctas, int x) {
  return total * x / ctas;
}

// ------------------------------------------------------------ per-type pieces

template <typename T, int D>
struct Shape {
  static constexpr int kRowBytes = D * static_cast<int>(sizeof(T));
  static constexpr int kChunks = kRowBytes / 16;  // 16-byte chunks per row
  static constexpr int kHalf = kTile * kRowBytes;  // bytes of a half tile
  // half tiles in a warp's ring: about 24 KB, so that two CTAs share an SM; at least 3
  static constexpr int kRing = kHalf <= 2048 ? 8 : kHalf == 4096 ? 6 : 3;
  static constexpr int kSteps = kChunks / 2;  // matrix steps over D (32 bytes each)
};

// Byte offset of 16-byte chunk `c` of row `r` in a half tile.  Chunks of eight
// consecutive rows at one c fall on eight different bank groups (ldmatrix);
// for f32 the order also keeps chunk pairs of four consecutive rows apart
// (the transposed 4-byte reads of V).
template <typename T, int D>
__device__ __forceinline__ int swizzled(int r, int c) {
  const int f = sizeof(T) == 4 ? ((r & 3) << 1 | (r >> 2 & 1)) : (r & 7);
  return r * Shape<T, D>::kRowBytes + ((c ^ f) << 4);
}

template <typename T, int D, int NT>
struct Warp;

// bf16: K fragments by ldmatrix, q fragments in registers.
template <int D, int NT>
struct Warp<__nv_bfloat16, D, NT> {
  using S = Shape<__nv_bfloat16, D>;
  static constexpr int kQSmem = 0;
  unsigned q[S::kSteps][NT][2];

  // row(n): q's row of column n of this warp's tile, or nullptr
  template <typename F>
  __device__ __forceinline__ void load_q(F row, void *, int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const __nv_bfloat16 *p = row(nt * 8 + lane / 4);
#pragma unroll
      for (int ks = 0; ks < S::kSteps; ++ks) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          q[ks][nt][b] = p ? *reinterpret_cast<const unsigned *>(p + ks * 16 + b * 8 + (lane & 3) * 2) : 0u;
      }
    }
  }

  __device__ __forceinline__ void scores(float (&s)[NT][4], unsigned k_tile, const void *, int lane) const {
    const int r = (lane & 7) + (lane >> 3 & 1) * 8;
#pragma unroll
    for (int ks = 0; ks < S::kSteps; ++ks) {
      unsigned a[4];
      ldmatrix_x4(a, k_tile + swizzled<__nv_bfloat16, D>(r, ks * 2 + (lane >> 4)));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16(s[nt], a, q[ks][nt][0], q[ks][nt][1]);
    }
  }

  // The B fragments of P^T from the score tile's layout: hi and lo halves.
  struct P {
    unsigned hi[NT][2], lo[NT][2];
    __device__ __forceinline__ P(const float (&p)[NT][4], int) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float x = p[nt][2 * b], y = p[nt][2 * b + 1];
          const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
          const __nv_bfloat162 l = __floats2bfloat162_rn(x - __low2float(h), y - __high2float(h));
          hi[nt][b] = movmatrix_trans(*reinterpret_cast<const unsigned *>(&h));
          lo[nt][b] = movmatrix_trans(*reinterpret_cast<const unsigned *>(&l));
        }
    }
  };

  // V^T fragment of 16 elements of D over the tile's 16 keys; keys outside [k0, k1) as zeros
  struct V {
    unsigned a[4];
    __device__ __forceinline__ V(unsigned v_tile, int md, int lane) {
      const int r = (lane & 7) + (lane >> 4) * 8;
      ldmatrix_x4_trans(a, v_tile + swizzled<__nv_bfloat16, D>(r, md * 2 + (lane >> 3 & 1)));
    }
    __device__ __forceinline__ void keep(int k0, int k1, int lane) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = h * 8 + (lane & 3) * 2;
        const unsigned m = (key >= k0 && key < k1 ? 0xffffu : 0u) | (key + 1 >= k0 && key + 1 < k1 ? 0xffff0000u : 0u);
        a[h * 2] &= m;
        a[h * 2 + 1] &= m;
      }
    }
    __device__ __forceinline__ void mma(float (&c)[4], const P &p, int nt) const {
      mma_bf16(c, a, p.hi[nt][0], p.hi[nt][1]);
      mma_bf16(c, a, p.lo[nt][0], p.lo[nt][1]);
    }
  };
};

// f32: three TF32 products of split operands; q in shared memory.
template <int D, int NT>
struct Warp<float, D, NT> {
  using S = Shape<float, D>;
  static constexpr int kQRow = D + 4;
  static constexpr int kQSmem = NT * 8 * kQRow * 4;

  template <typename F>
  __device__ __forceinline__ void load_q(F row, void *q_smem, int) {
    float *qs = static_cast<float *>(q_smem);
    for (int i = threadIdx.x; i < NT * 8 * D; i += kThreads) {
      const float *p = row(i / D);
      qs[i / D * kQRow + i % D] = p ? p[i % D] : 0.0f;
    }
  }

  __device__ __forceinline__ void scores(float (&s)[NT][4], unsigned k_tile, const void *q_smem, int lane) const {
    const float *qs = static_cast<const float *>(q_smem) + (lane / 4) * kQRow + (lane & 3);
    const int r = (lane & 7) + (lane >> 3 & 1) * 8;
#pragma unroll 4
    for (int ks = 0; ks < S::kSteps; ++ks) {
      unsigned a[4], hi[4], lo[4];
      ldmatrix_x4(a, k_tile + swizzled<float, D>(r, ks * 2 + (lane >> 4)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Tf32Pair x(__uint_as_float(a[i]));
        hi[i] = x.hi;
        lo[i] = x.lo;
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const Tf32Pair b0(qs[nt * 8 * kQRow + ks * 8]), b1(qs[nt * 8 * kQRow + ks * 8 + 4]);
        mma_tf32(s[nt], lo, b0.hi, b1.hi);
        mma_tf32(s[nt], hi, b0.lo, b1.lo);
        mma_tf32(s[nt], hi, b0.hi, b1.hi);
      }
    }
  }

  struct P {
    unsigned hi[NT][4], lo[NT][4];  // [key / 4]
    __device__ __forceinline__ P(const float (&p)[NT][4], int lane) {
      // value (key, row) is with lane (key % 8) * 4 + row / 2, in register key / 8 * 2 + row % 2
      const int src = (lane & 3) * 4 + (lane >> 3);
      const bool odd = lane >> 2 & 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float x = __shfl_sync(kFull, p[nt][(b >> 1) * 2], src + (b & 1) * 16);
          const float y = __shfl_sync(kFull, p[nt][(b >> 1) * 2 + 1], src + (b & 1) * 16);
          const Tf32Pair t(odd ? y : x);
          hi[nt][b] = t.hi;
          lo[nt][b] = t.lo;
        }
    }
  };

  struct V {
    unsigned hi[2][4], lo[2][4];  // two steps of 8 keys
    __device__ __forceinline__ V(unsigned v_tile, int md, int lane) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = h * 8 + (i >> 1) * 4 + (lane & 3), d = md * 16 + (i & 1) * 8 + lane / 4;
          float x;
          asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(x)
                       : "r"(v_tile + swizzled<float, D>(key, d >> 2) + (d & 3) * 4) : "memory");
          const Tf32Pair t(x);
          hi[h][i] = t.hi;
          lo[h][i] = t.lo;
        }
    }
    __device__ __forceinline__ void keep(int k0, int k1, int lane) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = h * 8 + (i >> 1) * 4 + (lane & 3);
          if (key < k0 || key >= k1) hi[h][i] = lo[h][i] = 0u;
        }
    }
    __device__ __forceinline__ void mma(float (&c)[4], const P &p, int nt) const {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_tf32(c, lo[h], p.hi[nt][2 * h], p.hi[nt][2 * h + 1]);
        mma_tf32(c, hi[h], p.lo[nt][2 * h], p.lo[nt][2 * h + 1]);
        mma_tf32(c, hi[h], p.hi[nt][2 * h], p.hi[nt][2 * h + 1]);
      }
    }
  };
};

template <typename T, int D, int NT>
constexpr int smem_bytes() {
  return kWarps * Shape<T, D>::kRing * Shape<T, D>::kHalf + Warp<T, D, NT>::kQSmem;
}

// ------------------------------------------------------------ the main kernel

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads) gdn_attn_paged_kernel(const __grid_constant__ Call c) {
  using S = Shape<T, D>;
  using W = Warp<T, D, NT>;
  constexpr int kRows = NT * 8;
  constexpr int kJoinRow = D + 4;  // padded row of the join area
  static_assert(kWarps * kRows * kJoinRow * 4 <= kWarps * S::kRing * S::kHalf, "the join area lies in the rings");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[kWarps], s_total, s_offset;
  __shared__ uint32_t s_seq;
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ int s_bad[kWarps];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char *ring = smem + warp * S::kRing * S::kHalf;
  const unsigned ring_at = smem_u32(ring);
  float *join = reinterpret_cast<float *>(smem);
  void *q_smem = smem + kWarps * S::kRing * S::kHalf;

  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");

  // This CTA's share of the units: the prefix sum of the requests' units, a
  // contiguous run of requests per thread.
  const uint32_t per = (c.n_seqs + kThreads - 1) / kThreads;
  const uint32_t s_first = min(tid * per, c.n_seqs), s_last = min(s_first + per, c.n_seqs);
  long long mine = 0;
  bool bad = false;
  for (uint32_t s = s_first; s < s_last; ++s) {
    const Request r = request<kRows>(c, s);
    mine += r.units(c);
    bad |= r.bad;
  }
  long long inc = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(kFull, inc, d);
    if (lane >= d) inc += x;
  }
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  before += inc - mine;
  if (bad && blockIdx.x == 0) report(GDN_DEVICE_BAD_REQUEST);
  const int ctas = static_cast<int>(min(total, static_cast<long long>(gridDim.x)));
  const int cta = blockIdx.x;
  if (tid == 0) c.meta[cta] = make_int4(0, 0, 0, -1);
  if (cta >= ctas) return;
  const long long u0 = share_start(total, ctas, cta), u1 = share_start(total, ctas, cta + 1);
  if (u0 >= before && u0 < before + mine) {
    long long at = before;
    for (uint32_t s = s_first; s < s_last; ++s) {
      const long long n = request<kRows>(c, s).units(c);
      if (u0 < at + n) {
        s_seq = s;
        s_offset = u0 - at;
        break;
      }
      at += n;
    }
  }
  __syncthreads();
  uint32_t seq = s_seq;
  long long in_seq = s_offset;  // units of the request before this point

  W w;
  for (long long u = u0; u < u1;) {
    Request r = request<kRows>(c, seq);
    while (in_seq >= r.units(c)) {  // next request with work
      in_seq = 0;
      if (++seq >= c.n_seqs) return;
      r = request<kRows>(c, seq);
    }
    const int item = static_cast<int>(in_seq / r.tiles);  // (head, row block) of the request
    const int tile0 = static_cast<int>(in_seq - static_cast<long long>(item) * r.tiles);
    const int tile1 = static_cast<int>(min(static_cast<long long>(r.tiles), tile0 + (u1 - u)));
    const int head = item / r.blocks, block = item - head * r.blocks;
    const int k0 = r.lo + tile0 * kUnit, k1 = min(r.len, r.lo + tile1 * kUnit);

    // Column n of the score tile is row block * kRows + n of the item: token row / group, query head row % group.
    const int rows = r.tokens * static_cast<int>(c.group);
    auto q_row = [&](int n) -> const T * {
      const int row = block * kRows + n;
      if (row >= rows) return nullptr;
      const int t = c.group_div.div(row);
      return static_cast<const T *>(c.q) + static_cast<int64_t>(r.t0 + t) * c.q_stride +
             (static_cast<int64_t>(head) * c.group + (row - t * static_cast<int>(c.group))) * D;
    };
    w.load_q(q_row, q_smem, lane);
    // the last key each of this lane's columns sees
    int last[NT][2], token[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = min(block * kRows + nt * 8 + (lane & 3) * 2 + j, rows - 1);
        token[nt][j] = c.group_div.div(row);
        last[nt][j] = r.len - r.tokens + token[nt][j];
      }
    const int t_first = c.group_div.div(block * kRows), t_last = c.group_div.div(min(block * kRows + kRows, rows) - 1);
    // keys in [all0, all1) are seen by every row of the block
    const int all1 = r.len - r.tokens + t_first + 1;
    const int all0 = c.window ? r.len - r.tokens + t_last + 1 - static_cast<int>(min(c.window, 0x3fffffffu)) : 0;
    if (W::kQSmem) __syncthreads();

    float acc[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.0f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.0f;
    }

    // This warp's tiles: keys k0 + 16 (warp + 4 i).
    const int first = k0 + kTile * warp;
    const int n_tiles = first < k1 ? (k1 - first + kUnit - 1) / kUnit : 0;
    const int32_t *table = c.table + static_cast<uint64_t>(seq) * c.max_pages;
    // Lane i < 16 (and i + 16) looks up tile row i: page number now, a tile ahead of its use.
    auto page_of = [&](int i) -> int {
      const int key = first + i * kUnit + (lane & 15);
      return i < n_tiles && key < k1 ? table[c.page_div.div(key)] : 0;
    };
    int page = page_of(0);
    bool bad_page = false;
    long long row_at = -1;  // element offset of this lane's row of the tile being fetched; -1: zeros
    auto fetch = [&](int h) {  // half tile h: K of tile h / 2, or V
      const int i = h >> 1;
      if (i < n_tiles) {
        if (!(h & 1)) {
          const int key = first + i * kUnit + (lane & 15);
          const int j = c.page_div.div(key);
          row_at = -1;
          if (key < k1) {
            if (static_cast<uint32_t>(page) < c.n_pages)
              row_at = page * c.page_stride + head * c.head_stride + static_cast<int64_t>(key - j * static_cast<int>(c.page_size)) * c.slot_stride;
            else
              bad_page = true;
          }
          page = page_of(i + 1);
        }
        const T *base = static_cast<const T *>(h & 1 ? c.v : c.k);
        const unsigned to = ring_at + (h % S::kRing) * S::kHalf;
#pragma unroll
        for (int x = 0; x < kTile * S::kChunks / 32; ++x) {
          const int at = x * 32 + lane, row = at / S::kChunks, ch = at % S::kChunks;
          const long long off = __shfl_sync(kFull, row_at, row);
          cp_async_16_or_zero(to + swizzled<T, D>(row, ch), base + (off < 0 ? 0 : off) + ch * (16 / static_cast<int>(sizeof(T))), off >= 0);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int h = 0; h < S::kRing - 1; ++h) fetch(h);

    unsigned slot = 0;
    for (int i = 0; i < n_tiles; ++i) {
      const int key0 = first + i * kUnit;
      // scores
      fetch(2 * i + S::kRing - 1);
      cp_async_wait<S::kRing - 1>();
      __syncwarp();
      float s[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
      w.scores(s, ring_at + slot * S::kHalf, q_smem, lane);
      slot = slot + 1 == S::kRing ? 0 : slot + 1;
      const bool edge = key0 + kTile > min(all1, k1) || key0 < all0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = s[nt][j] * c.scale_log2, y = s[nt][j + 2] * c.scale_log2;
          if (edge) {
            const int ka = key0 + lane / 4, kb = ka + 8;
            const int hi = min(last[nt][j], k1 - 1);
            const long long lo = c.window ? static_cast<long long>(last[nt][j]) - c.window : -1;
            if (ka > hi || ka <= lo) x = -INFINITY;
            if (kb > hi || kb <= lo) y = -INFINITY;
          }
          float top = fmaxf(x, y);
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
          top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
          top = fmaxf(top, m[nt][j]);
          const float base = top == -INFINITY ? 0.0f : top;  // nothing seen yet: exp2(-inf) = 0
          f[j] = exp2f(m[nt][j] - base);
          m[nt][j] = top;
          s[nt][j] = exp2f(x - base);
          s[nt][j + 2] = exp2f(y - base);
          l[nt][j] = l[nt][j] * f[j] + (s[nt][j] + s[nt][j + 2]);
        }
        if (__any_sync(kFull, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
          for (int md = 0; md < D / 16; ++md) {
            acc[md][nt][0] *= f[0];
            acc[md][nt][1] *= f[1];
            acc[md][nt][2] *= f[0];
            acc[md][nt][3] *= f[1];
          }
        }
      }
      const typename W::P p(s, lane);
      // output
      __syncwarp();
      fetch(2 * i + S::kRing);
      cp_async_wait<S::kRing - 1>();
      __syncwarp();
      const unsigned v_tile = ring_at + slot * S::kHalf;
      slot = slot + 1 == S::kRing ? 0 : slot + 1;
      if (!edge || t_first == t_last) {
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          typename W::V v(v_tile, md, lane);
          if (edge) v.keep(all0 - key0, min(all1, k1) - key0, lane);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) v.mma(acc[md][nt], p, nt);
        }
      } else {
        // Tokens see different keys of this tile.  A key that a token does not see must not reach its
        // row even as 0 * v (v may be infinite or NaN), so each token's columns take the product with
        // V's unseen keys cut out.
#pragma unroll 1
        for (int t = t_first; t <= t_last; ++t) {
          const int hi = r.len - r.tokens + t + 1 - key0;
          const int lo = c.window ? hi - static_cast<int>(min(c.window, 0x3fffffffu)) : -1;
#pragma unroll
          for (int md = 0; md < D / 16; ++md) {
            typename W::V v(v_tile, md, lane);
            v.keep(lo, min(hi, k1 - key0), lane);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              v.mma(y, p, nt);
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (token[nt][j & 1] == t) acc[md][nt][j] += y[j];
            }
          }
        }
      }
      __syncwarp();
    }
    cp_async_wait<0>();

    // Join the four warps.
    bad_page = __any_sync(kFull, bad_page);
    if (lane == 0) s_bad[warp] = bad_page;
    __syncthreads();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nt * 8 + (lane & 3) * 2 + j;
        float x = l[nt][j];
        x += __shfl_xor_sync(kFull, x, 4);
        x += __shfl_xor_sync(kFull, x, 8);
        x += __shfl_xor_sync(kFull, x, 16);
        if (lane < 4) {
          s_m[warp][row] = m[nt][j];
          s_l[warp][row] = x;
        }
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          join[(warp * kRows + row) * kJoinRow + md * 16 + lane / 4] = acc[md][nt][j];
          join[(warp * kRows + row) * kJoinRow + md * 16 + lane / 4 + 8] = acc[md][nt][j + 2];
        }
      }
    __syncthreads();
    const bool whole = tile0 == 0 && tile1 == r.tiles;
    const int part_slot = 2 * cta + (u == u0 ? 0 : 1);
    const bool poison = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];  // rows over a page that does not exist are NaN
    if (poison && tid == 0) report(GDN_DEVICE_BAD_PAGE);
    for (int x = tid; x < kRows * D; x += kThreads) {
      const int row = x / D, d = x % D, item_row = block * kRows + row;
      if (item_row >= rows) break;
      float top = s_m[0][row];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) top = fmaxf(top, s_m[i][row]);
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f, den = 0.0f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float f = exp2f(s_m[i][row] - base);
        sum += f * join[(i * kRows + row) * kJoinRow + d];
        den += f * s_l[i][row];
      }
      if (poison) sum = den = NAN;
      if (whole) {
        const int t = c.group_div.div(item_row);
        // a row that sees no key is zero; one whose visible scores are all -inf is 0 / 0
        const bool empty = r.len - r.tokens + t < 0;
        T *o = static_cast<T *>(c.out) + static_cast<int64_t>(r.t0 + t) * c.out_stride +
               (static_cast<int64_t>(head) * c.group + (item_row - t * static_cast<int>(c.group))) * D + d;
        Act<T>::put(o, empty && !poison ? 0.0f : sum / den);
      } else {
        c.part[(static_cast<size_t>(part_slot) * kRows + row) * D + d] = sum;
        if (d == 0) c.part_ml[static_cast<size_t>(part_slot) * kRows + row] = make_float2(top, den);
      }
    }
    if (!whole && tile0 == 0 && tid == 0) {
      const long long end = u + r.tiles - 1;  // the item's last unit
      c.meta[cta] = make_int4(static_cast<int>(seq), item, static_cast<int>(((end + 1) * ctas - 1) / total), part_slot);
    }
    u += tile1 - tile0;
    in_seq += tile1 - tile0;
    __syncthreads();
  }
}

// ------------------------------------------------------------ the join

// CTA (x, y): row y of the item that begins in main CTA x and goes on in later
// ones.  Each warp takes every fourth of the item's parts.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kJoinWarps) gdn_attn_join_kernel(const __grid_constant__ Call c) {
  constexpr int kRows = NT * 8, kPer = D / 32;
  __shared__ float s_acc[kJoinWarps][D], s_den[kJoinWarps];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int4 meta = c.meta[blockIdx.x];
  if (meta.w < 0) return;
  const Request r = request<kRows>(c, meta.x);
  const int head = meta.y / r.blocks, block = meta.y - head * r.blocks;
  const int row = blockIdx.y, item_row = block * kRows + row;
  if (item_row >= r.tokens * static_cast<int>(c.group)) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x0 = blockIdx.x, n = meta.z - x0 + 1;
  auto slot = [&](int i) { return static_cast<size_t>(i == 0 ? meta.w : 2 * (x0 + i)) * kRows + row; };

  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, c.part_ml[slot(i)].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, d));
  const float base = top == -INFINITY ? 0.0f : top;
  float acc[kPer] = {}, den = 0.0f;
#pragma unroll 4
  for (int i = warp; i < n; i += kJoinWarps) {
    const float2 ml = c.part_ml[slot(i)];
    const float f = exp2f(ml.x - base);
    den += f * ml.y;
    const float *src = c.part + slot(i) * D + lane;
#pragma unroll
    for (int j = 0; j < kPer; ++j) acc[j] += f * src[j * 32];
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) s_acc[warp][j * 32 + lane] = acc[j];
  if (lane == 0) s_den[warp] = den;
  __syncthreads();
  den = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) den += s_den[w];
  const int t = c.group_div.div(item_row);
  T *o = static_cast<T *>(c.out) + static_cast<int64_t>(r.t0 + t) * c.out_stride +
         (static_cast<int64_t>(head) * c.group + (item_row - t * static_cast<int>(c.group))) * D;
  const bool empty = r.len - r.tokens + t < 0;
  for (int d = threadIdx.x; d < D; d += 32 * kJoinWarps) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) sum += s_acc[w][d];
    Act<T>::put(o + d, empty && !isnan(den) ? 0.0f : sum / den);
  }
}

// ------------------------------------------------------------ host

template <typename T, int D, int NT>
constexpr int ctas_per_sm() {
  const int by_smem = 227 * 1024 / (smem_bytes<T, D, NT>() + 2048);
  return by_smem < 1 ? 1 : by_smem > 4 ? 4 : by_smem;
}

int row_tiles(const gdn_attn_params &p) {
  const uint64_t window = (p.n_tokens + static_cast<uint64_t>(p.n_seqs) - 1) / p.n_seqs;
  return window * (p.n_q_heads / p.n_kv_heads) <= 8 ? 1 : 2;
}

// calls f(type, D, NT) with the call's compile-time values
template <typename F>
auto dispatch(const gdn_attn_params &p, F f) {
  auto by_rows = [&](auto t, auto d) {
    return row_tiles(p) == 1 ? f(t, d, std::integral_constant<int, 1>{}) : f(t, d, std::integral_constant<int, 2>{});
  };
  auto by_dim = [&](auto t) {
    return p.head_dim == 64    ? by_rows(t, std::integral_constant<int, 64>{})
           : p.head_dim == 128 ? by_rows(t, std::integral_constant<int, 128>{})
                               : by_rows(t, std::integral_constant<int, 256>{});
  };
  return p.dtype == GDN_DTYPE_BF16 ? by_dim(__nv_bfloat16{}) : by_dim(float{});
}

size_t part_floats(int ctas, int rows, int d) { return static_cast<size_t>(2) * ctas * rows * d; }

}  // namespace

size_t attn_workspace_bytes(const gdn_attn_params &p) {
  return dispatch(p, [&](auto t, auto d, auto nt) {
    constexpr int ctas = kSms * ctas_per_sm<decltype(t), d(), nt()>();
    return part_floats(ctas, nt() * 8, d()) * 4 + static_cast<size_t>(2) * ctas * nt() * 8 * sizeof(float2) +
           ctas * sizeof(int4);
  });
}

cudaError_t launch_attn_paged(const AttnArgs &a, cudaStream_t stream) {
  const gdn_attn_params &p = a.p;
  Call c;
  c.q = a.q;
  c.k = a.k_cache;
  c.v = a.v_cache;
  c.table = a.block_table;
  c.kv_lens = a.kv_lens;
  c.token_start = a.token_start;
  c.out = a.output;
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
  return dispatch(p, [&](auto t, auto d, auto nt) {
    using T = decltype(t);
    constexpr int D = d(), NT = nt(), ctas = kSms * ctas_per_sm<T, D, NT>(), smem = smem_bytes<T, D, NT>();
    // widest alignment first: sums, (maximum, sum) pairs, item records
    c.meta = static_cast<int4 *>(a.workspace);
    c.part = reinterpret_cast<float *>(c.meta + ctas);
    c.part_ml = reinterpret_cast<float2 *>(c.part + part_floats(ctas, NT * 8, D));
    cudaError_t e = cudaFuncSetAttribute(gdn_attn_paged_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    gdn_attn_paged_kernel<T, D, NT><<<ctas, kThreads, smem, stream>>>(c);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // The join may be set up while the main kernel still runs; it waits for its end before it reads.
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas, NT * 8);
    cfg.blockDim = dim3(32 * kJoinWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, gdn_attn_join_kernel<T, D, NT>, static_cast<const Call>(c));
  });
}

cudaError_t attn_paged_status(unsigned int *bits, bool reset, cudaStream_t stream) {
  return read_paged_status(bits, reset, stream);
}

}  // namespace gdn
