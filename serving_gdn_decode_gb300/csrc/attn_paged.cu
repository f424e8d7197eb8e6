// Attention of each request's newest tokens over its paged key-value cache
// (gdn_attn_paged): out = sum_j softmax_j(scale q.k_j) v_j over the keys a
// token sees, for windows of one token (decode) to a few (verification).
//
// What bounds it.  Every cached key and value is read once and used for
// group x window rows, 2 to about 100 flops a byte in bf16: HBM bounds it, far
// from the tensor cores' rate, so the kernel is built around keeping loads in
// flight.  A token's rows sit on the N side of the matrix instruction (S^T = K
// Q^T, O^T = V^T P^T): N is 8 there, so a group of 1 to 8 query heads wastes
// the least, and accumulators stay in registers.  The warp-level mma.sync
// serves this (14 % of the tensor cycles at 4 rows per key head); a tcgen05 tile
// would put 128 keys on the M side for the same 8 columns and pay tensor-memory
// round trips between two tiny products.  Past 32 rows per key head that turns:
// there the warp-level instructions and their operand reads bound the kernel.
//
// Measured on a GB300, back to back over three sets of buffers, as shares of the
// measured copy bandwidth (6783 GB/s): 64 requests of up to 4096 keys, 32/8 heads
// of 128, bf16: 81 us, 0.90; 256 requests, 48/8 heads: 308 us, 0.98; one request
// of 200003 keys, 32/4 heads: 68 us, 0.89; 16 rows per key head: 0.91; 17 to 24 rows
// at head_dim 256: 0.60 to 0.71; 32 rows: 0.58 to 0.82; 56 rows: 0.43 to 0.58; f32 with
// 2 to 8 rows per key head: 0.87 to 0.97, with one, heads of 64: 0.71.  Below
// about 100 MB of cache the fixed part shows: 2.5 us of launch, 3 us until the
// first products (lengths, page numbers and keys are three dependent reads), and
// 3 us for the join.
//
// Split over the length.  The work of a call is a list of units: 64 keys, and
// two units for an item's begin and end (an item is a request's key head and
// block of rows; without the two, CTAs with many short items finished 25 %
// late).  The lengths are on the device, so every CTA takes the prefix sum of
// the requests' units and then the same share of the whole list, whatever the
// lengths are.  A share may begin and end inside an item: such ends leave
// unnormalised sums with their running maximum in the workspace (at most two per
// CTA), and a second launch joins them; an item that lies in one CTA goes
// straight to the output.  No atomics: the order of every sum is fixed by the
// sizes.
//
// Inside a CTA each key group (a warp, or with more rows several warps that share
// a ring) takes every KW-th tile of the item with a softmax state of its own, and
// the groups are joined at the item's end; so the main loop has no barrier between
// groups.  A group feeds itself through a ring of half tiles (16 or 32 rows of K,
// then the same rows of V) with 16-byte asynchronous copies, which follow any page
// size, stride and tile edge; 80 to 190 KB per SM are on their way.  The feed runs
// on into the next items, so that the ring does not drain between them.
//
// Precision.  f32: each operand is split in two TF32 halves and three products
// are taken, so a product is good to 2^-20.  bf16: K, V and q are exact in the
// products; the probabilities are split in two bf16 halves (two products instead
// of one: bytes, not products, bound the kernel), each off by 2^-16 of itself at
// most, to either side: a 256th of what the result's one rounding, at the end,
// may take.  The maximum, the sums and all accumulators are
// f32; a tile's sum is added to the running one outside the tensor cores, but for
// the short sums of kShortKeys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "device_io.cuh"
#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr int kSub = 16;   // keys of a matrix tile
constexpr int kUnit = 64;  // keys per unit of work
constexpr int kMostTile = 32;  // largest tile of a key group
constexpr int kItemUnits = 2;  // what an item's begin and end cost beside its keys, in units
constexpr int kSms = 152;
constexpr int kJoinWarps = 8;

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLowest = -3.402823466e38f;  // the lowest finite f32

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
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// c += a (16 x 16) b (16 x 8), bf16
__device__ __forceinline__ void mma_bf16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c += a (16 x 8) b (8 x 8), TF32
__device__ __forceinline__ void mma_tf32(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + lo up to 2^-23 |x|, both with TF32's 10 mantissa bits: hi is x rounded to nearest (a carry into the
// exponent is the next binade), lo the exact rest, at most 12 bits, of which the matrix instruction reads 11; the cut
// leans to neither side since the rest has either sign.  From 3.4026e38 on the carry would make hi an infinity and lo
// the other one; with TOP hi stops at TF32's largest value and the rest, an infinity or a NaN too, is in lo.
template <bool TOP>
struct Tf32Pair {
  unsigned hi, lo;
  __device__ __forceinline__ explicit Tf32Pair(float x) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    if constexpr (TOP) {
      float h;  // the smaller magnitude, with x's sign
      asm("min.xorsign.abs.f32 %0, %1, %2;\n" : "=f"(h) : "f"(__uint_as_float(hi)), "f"(3.40116213421e38f));
      hi = __float_as_uint(h);
    }
    lo = __float_as_uint(x - __uint_as_float(hi));
  }
};
// x = hi + lo, hi being x cut to TF32, which is finite where x is, lo the exact rest, at most 13 bits: rounded to
// nearest by the addition and the instruction's cut (ROUND: up to 2^-22 |x|), or cut (up to 2^-21 |x|, 2^-23 on
// average, towards zero; f32's largest value would round up to an infinity).  An infinity or a NaN is in hi, a NaN whose
// payload is in its 13 low bits alone as an infinity.  Beside the other split's lo, which has either sign, the product
// lo * lo that is left out is below 2^-21 and leans to neither side.
template <bool ROUND>
struct Tf32Cut {
  unsigned hi, lo;
  __device__ __forceinline__ explicit Tf32Cut(float x) {
    hi = __float_as_uint(x) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi)) + (ROUND ? 0x1000u : 0u);
  }
};

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

// ------------------------------------------------------------ per-type pieces

// KT: matrix tiles of 16 keys in a tile, the step of a key group.
template <typename T, int D, int KT>
struct Shape {
  static constexpr int kTile = kSub * KT;
  static constexpr int kRowBytes = D * static_cast<int>(sizeof(T));
  static constexpr int kChunks = kRowBytes / 16;   // 16-byte chunks per row
  static constexpr int kHalf = kTile * kRowBytes;  // bytes of a half tile
  // half tiles in a CTA's rings together
  static constexpr int kSlots16 = kRowBytes == 128   ? 32
                                  : kRowBytes == 256 ? (sizeof(T) == 4 ? 12 : 20)
                                  : kRowBytes == 512 ? (sizeof(T) == 4 ? 20 : 24)
                                                     : 12;
  static constexpr int kSlots = kSlots16 / KT;
  static constexpr int kSteps = kChunks / 2;       // matrix steps over D (32 bytes each)
};

// A half tile in shared memory: row r's chunk c lies at r * kRowBytes +
// ((c ^ order(r)) << 4).  order permutes the three low bits, so that one chunk
// of eight consecutive rows falls on eight different bank groups (ldmatrix);
// for f32 it also keeps two neighbouring chunks of four consecutive rows apart
// (the transposed 4-byte reads of V).  order(x ^ y) = order(x) ^ order(y): a
// lane's offset for a step is its offset for step 0 with a constant XORed in.
template <typename T>
__device__ __host__ constexpr int order(int r) {
  return sizeof(T) == 4 ? ((r & 3) << 1 | (r >> 2 & 1)) : (r & 7);
}
template <typename T, int D>
__device__ __forceinline__ constexpr int swizzled(int r, int c) {
  return r * D * static_cast<int>(sizeof(T)) + ((c ^ order<T>(r)) << 4);
}

// NT: 8-row tiles of a warp.  RW: warps that share a ring, each with rows of its
// own.  A CTA has WARPS warps, WARPS / RW key groups with a ring each.
template <typename T, int D, int NT, int RW>
struct Warp;

// bf16: K and V fragments by ldmatrix, q fragments in registers.
template <int D, int NT, int RW>
struct Warp<__nv_bfloat16, D, NT, RW> {
  using S = Shape<__nv_bfloat16, D, 1>;
  static constexpr int kQSmem = 0;
  unsigned q[S::kSteps][NT][2];
  unsigned k_at[4], v_at[4];  // this lane's offsets in a half tile for steps 0-3; step + 4: 128 bytes on

  __device__ __forceinline__ Warp(int lane, int) {
    const int rk = (lane & 7) + (lane >> 3 & 1) * 8, rv = (lane & 7) + (lane >> 4) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      k_at[i] = swizzled<__nv_bfloat16, D>(rk, i * 2 + (lane >> 4));
      v_at[i] = swizzled<__nv_bfloat16, D>(rv, i * 2 + (lane >> 3 & 1));
    }
  }

  // row(n): q's row of column n of the CTA's block, or nullptr; this warp's begin at row0
  template <typename F>
  __device__ __forceinline__ void load_q(F row, void *, int lane, int row0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const __nv_bfloat16 *p = row(row0 + nt * 8 + lane / 4);
#pragma unroll
      for (int ks = 0; ks < S::kSteps; ++ks) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          q[ks][nt][b] = p ? *reinterpret_cast<const unsigned *>(p + ks * 16 + b * 8 + (lane & 3) * 2) : 0u;
      }
    }
  }

  // s = K Q^T of the tile's 16 keys; several chains of products, for their latency
  __device__ __forceinline__ void scores(float (&s)[NT][4], unsigned k_tile, const void *) const {
    constexpr int kChains = NT == 1 ? 4 : 2;
    float t[kChains][NT][4];
#pragma unroll
    for (int i = 0; i < kChains; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) t[i][nt][0] = t[i][nt][1] = t[i][nt][2] = t[i][nt][3] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < S::kSteps; ++ks) {
      unsigned a[4];
      ldmatrix_x4(a, k_tile + k_at[ks & 3] + (ks >> 2) * 128);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) mma_bf16(t[ks % kChains][nt], a, q[ks][nt][0], q[ks][nt][1]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[nt][j] = t[0][nt][j] + t[1][nt][j];
        if (kChains == 4) s[nt][j] += t[kChains - 2][nt][j] + t[kChains - 1][nt][j];
      }
  }

  // The B fragments of P^T from the score tile's layout: hi and lo halves.
  struct P {
    unsigned hi[NT][2], lo[NT][2];
    __device__ __forceinline__ void take(const float (&p)[NT][4], int) {
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

  // V^T fragment of 16 elements of D over the tile's 16 keys
  struct V {
    unsigned a[4];
    __device__ __forceinline__ V(const Warp &w, unsigned v_tile, int md) {
      ldmatrix_x4_trans(a, v_tile + w.v_at[md & 3] + (md >> 2) * 128);
    }
    // keys outside [k0, k1) as zeros
    __device__ __forceinline__ void keep(int k0, int k1, int lane) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int key = h * 8 + (lane & 3) * 2;
        const unsigned m = (key >= k0 && key < k1 ? 0xffffu : 0u) | (key + 1 >= k0 && key + 1 < k1 ? 0xffff0000u : 0u);
        a[h * 2] &= m;
        a[h * 2 + 1] &= m;
      }
    }
    // m: the largest magnitudes so far, as bits
    __device__ __forceinline__ void largest(unsigned &m) const {
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, a[i] & 0x7fff7fffu);
    }
    static __device__ __forceinline__ bool finite(unsigned m) { return (m & 0xffffu) < 0x7f80u && (m >> 16) < 0x7f80u; }
    // y += V^T P^T, the sum of one tile
    __device__ __forceinline__ void mma(float (&y)[4], const P &p, int nt) const {
      mma_bf16(y, a, p.lo[nt][0], p.lo[nt][1]);
      mma_bf16(y, a, p.hi[nt][0], p.hi[nt][1]);
    }
  };
};

// f32: three TF32 products of split operands; q's halves in shared memory.
// As the output's sums, those of a score are taken outside the tensor cores: a
// product's sum starts at zero, over 32 elements of D, and is added in f32.
template <int D, int NT, int RW>
struct Warp<float, D, NT, RW> {
  using S = Shape<float, D, 1>;
  // Heads of 64, 16/16, 24 requests, window 1000: 33.5 us with Tf32Pair, 36.4 with Tf32Cut (whose form spills);
  // 64 requests up to 4096 keys, 32/8 heads of 128: 186 and 175; 8/4 heads of 256: 174 and 156.
  using KeyHalves = std::conditional_t<D == 64, Tf32Pair<true>, Tf32Cut<true>>;
  using ValueHalves = std::conditional_t<D == 64, Tf32Pair<true>, Tf32Cut<false>>;
  static constexpr int kQRow = 2 * D + 8;  // (hi, lo) pairs, padded
  static constexpr int kQSmem = RW * NT * 8 * kQRow * 4;
  unsigned k_at[4], v_at[8], q_at;

  __device__ __forceinline__ Warp(int lane, int row0) {
    const int rk = (lane & 7) + (lane >> 3 & 1) * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) k_at[i] = swizzled<float, D>(rk, i * 2 + (lane >> 4));
    // key (i & 1) * 4 + lane % 4, element (i >> 1) * 8 + lane / 4
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v_at[i] = swizzled<float, D>((i & 1) * 4 + (lane & 3), (i >> 1) * 2 + (lane >> 4)) + (lane >> 2 & 3) * 4;
    q_at = (row0 + lane / 4) * kQRow + (lane & 3) * 2;
  }

  template <typename F>
  __device__ __forceinline__ void load_q(F row, void *q_smem, int, int) {
    // four elements a time, all of a thread's on their way before the first is split
    constexpr int kFours = RW * NT * 8 * D / 4, kMine = kFours / 128;
    float x[kMine][4];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int at = threadIdx.x + i * 128, col = at % (D / 4) * 4;
      const float *p = row(at / (D / 4));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = p ? p[col + e] : 0.0f;
    }
    uint4 *qs = static_cast<uint4 *>(q_smem);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int at = threadIdx.x + i * 128, col = at % (D / 4) * 4;
      const Tf32Pair<true> a(x[i][0]), b(x[i][1]), c(x[i][2]), d(x[i][3]);
      uint4 *to = qs + (at / (D / 4) * kQRow + col * 2) / 4;
      to[0] = make_uint4(a.hi, a.lo, b.hi, b.lo);
      to[1] = make_uint4(c.hi, c.lo, d.hi, d.lo);
    }
  }

  __device__ __forceinline__ void scores(float (&s)[NT][4], unsigned k_tile, const void *q_smem) const {
    const unsigned *qs = static_cast<const unsigned *>(q_smem) + q_at;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll(S::kSteps / 4 > 2 ? 2 : S::kSteps / 4)
    for (int k4 = 0; k4 < S::kSteps / 4; ++k4) {
      float t[NT][4], e[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) t[nt][j] = e[nt][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        unsigned a[4], lo[4];
        ldmatrix_x4(a, k_tile + k_at[i] + k4 * 128);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const KeyHalves x(__uint_as_float(a[j]));
          a[j] = x.hi;
          lo[j] = x.lo;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 b0 = *reinterpret_cast<const uint2 *>(qs + nt * 8 * kQRow + (k4 * 4 + i) * 16);
          const uint2 b1 = *reinterpret_cast<const uint2 *>(qs + nt * 8 * kQRow + (k4 * 4 + i) * 16 + 8);
          mma_tf32(t[nt], a, b0.x, b1.x);
          mma_tf32(e[nt], lo, b0.x, b1.x);
          mma_tf32(e[nt], a, b0.y, b1.y);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nt][j] += t[nt][j] + e[nt][j];
    }
  }

  struct P {
    unsigned hi[NT][4], lo[NT][4];  // [key / 4]
    __device__ __forceinline__ void take(const float (&p)[NT][4], int lane) {
      // value (key, row) is with lane (key % 8) * 4 + row / 2, in register key / 8 * 2 + row % 2
      const int src = (lane & 3) * 4 + (lane >> 3);
      const bool odd = lane >> 2 & 1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float x = __shfl_sync(kFull, p[nt][(b >> 1) * 2], src + (b & 1) * 16);
          const float y = __shfl_sync(kFull, p[nt][(b >> 1) * 2 + 1], src + (b & 1) * 16);
          const Tf32Pair<false> t(odd ? y : x);  // at most 2^8
          hi[nt][b] = t.hi;
          lo[nt][b] = t.lo;
        }
    }
  };

  struct V {
    unsigned hi[2][4], lo[2][4];  // two steps of 8 keys
    __device__ __forceinline__ V(const Warp &w, unsigned v_tile, int md) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // register i: key (i >> 1) * 4 + lane % 4 of the step, element (i & 1) * 8 + lane / 4 of the 16
          float x;
          asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(x)
                       : "r"(v_tile + w.v_at[(md & 1) * 4 + (i & 1) * 2 + (i >> 1)] + (md >> 1) * 128 + h * 8 * S::kRowBytes)
                       : "memory");
          const ValueHalves t(x);
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
    __device__ __forceinline__ void largest(unsigned &m) const {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(hi[h][i] & 0x7fffffffu, lo[h][i] & 0x7fffffffu));
    }
    static __device__ __forceinline__ bool finite(unsigned m) { return m < 0x7f800000u; }
    __device__ __forceinline__ void mma(float (&y)[4], const P &p, int nt) const {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_tf32(y, lo[h], p.hi[nt][2 * h], p.hi[nt][2 * h + 1]);
        mma_tf32(y, hi[h], p.lo[nt][2 * h], p.lo[nt][2 * h + 1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) mma_tf32(y, hi[h], p.hi[nt][2 * h], p.hi[nt][2 * h + 1]);
    }
  };
};

// The join of a CTA's warps goes through shared memory in pieces of 8 rows x join_cols, rows padded so that a
// fragment's fall on different banks.
template <typename T, int D, int WARPS>
constexpr int join_cols() {
  return D < 256 || (sizeof(T) == 2 && WARPS == 4) ? D : 128;
}
template <typename T, int D, int WARPS>
constexpr int join_bytes() {
  return WARPS * 8 * (join_cols<T, D, WARPS>() + 4) * 4;
}
template <typename T, int D, int NT, int RW, int WARPS, int KT>
constexpr int smem_bytes() {
  return Shape<T, D, KT>::kSlots * Shape<T, D, KT>::kHalf + join_bytes<T, D, WARPS>() + Warp<T, D, NT, RW>::kQSmem;
}
// CTAs an SM holds: its shared memory, and registers enough for the accumulators
template <typename T, int D, int NT, int RW, int WARPS, int KT>
constexpr int ctas_per_sm() {
  const int by_smem = 227 * 1024 / (smem_bytes<T, D, NT, RW, WARPS, KT>() + 1024);  // + the static part
  const int by_regs = sizeof(T) == 4 && NT == 2 ? 2 : 3;
  return by_smem > by_regs ? by_regs : by_smem;
}

// The tensor cores cut the low bits of a running sum at every product, always towards zero: over n products a sum
// kept there leans by up to n 2^-24 of itself (6.9e-3 over 2^20 keys, measured).  So a tile's sum starts at zero and
// is added in f32, rounded to nearest.  That costs bf16 a few registers and the latency of a product, where there are
// few of either (64 requests up to 8192 keys, windows of 1 to 7, 8 heads of 128 per key head: 274 us, and 248 with the
// sums in the tensor cores; of 256: 288 and 276; 32 requests, windows of 1 to 4, 8 of 256: 65 and 61; heads of 64 and
// 32 rows: 237 and 229; heads of 128 with one row tile: equal).  There the part of an item that lies in a CTA keeps its
// sums in the tensor cores if it has at most kShortKeys keys per key group: 1024 products, 2^-14 of the sum, a 32nd of
// the result's rounding to bf16.  At 128 elements its edge tiles do not, for the registers.
constexpr int kShortKeys = 8192;
template <typename T, int D, int NT>
constexpr bool kKeepsShortSums = sizeof(T) == 2 && (D != 128 || NT > 1);

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

// ------------------------------------------------------------ the main kernel

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

template <typename T, int D, int NT, int RW, int WARPS, int KT>
__global__ void __launch_bounds__(32 * WARPS, (ctas_per_sm<T, D, NT, RW, WARPS, KT>())) gdn_attn_paged_kernel(const __grid_constant__ Call c) {
  using S = Shape<T, D, KT>;
  using W = Warp<T, D, NT, RW>;
  constexpr int kTile = S::kTile;
  constexpr int kJoinCols = join_cols<T, D, WARPS>(), kJoinRow = kJoinCols + 4;
  constexpr int kRows = RW * NT * 8;   // rows of a block
  constexpr int KW = WARPS / RW;       // key groups
  constexpr int kThreads = 32 * WARPS;
  constexpr int kStep = kTile * KW;    // keys from a group's tile to its next
  constexpr int kRing = S::kSlots / KW;
  static_assert(ctas_per_sm<T, D, NT, RW, WARPS, KT>() >= 1, "a CTA fits an SM's shared memory");
  static_assert(kRing <= 32, "a bit per slot");
  static_assert(sizeof(T) == 2 || WARPS == 4, "the f32 form loads q with 128 threads");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[WARPS], s_offset;
  __shared__ uint32_t s_seq;
  __shared__ float s_m[WARPS][NT * 8], s_l[WARPS][NT * 8];
  __shared__ int s_bad[WARPS];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kg = warp / RW, rg = warp % RW, row0 = rg * NT * 8;  // key group; rows of the block
  const unsigned ring = smem_u32(smem) + kg * kRing * S::kHalf;
  float *join = reinterpret_cast<float *>(smem + S::kSlots * S::kHalf);
  void *q_smem = smem + S::kSlots * S::kHalf + join_bytes<T, D, WARPS>();

  begin_in_order();

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
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += s_scan[w];
    total += s_scan[w];
  }
  before += inc - mine;
  if (bad && blockIdx.x == 0) report(GDN_DEVICE_BAD_REQUEST);
  const int ctas = static_cast<int>(min(total, static_cast<long long>(gridDim.x)));
  const int cta = blockIdx.x;
  if (tid == 0) c.splits[cta].slot = -1;
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

  // The ring's feed runs ahead of the products, across items: `f` is the item
  // that the next half tile belongs to, `f_i` its tile.
  Item<kRows, KW, kTile> f;
  f.seq = s_seq;
  f.in_seq = s_offset;
  f.r = request<kRows>(c, f.seq);
  Item<kRows, KW, kTile> it = f;
  long long f_u = u0;
  int f_i = 0, f_n = 0, f_head = 0;
  unsigned f_slot = 0;
  const int32_t *f_table = nullptr;
  bool f_value = false, f_any = false;
  unsigned bad_slots = 0;  // bit i: the K tile in slot i of the ring is not there (its page is none of the cache's), and
                           // is not wholly before the window: pages that the window has left may be given back
  int page = 0;          // the page of the next tile (of this lane's row of it), looked up a tile ahead
  long long row_at = 0;  // byte offset of the tile's first row (of this lane's row; -1: zeros) in the caches
  constexpr int kPer = S::kChunks >= 32 ? 1 : 32 / S::kChunks;  // rows one access of the warp covers
  constexpr int kAccesses = kTile * S::kChunks / 32 / RW;  // of this warp for a half tile
  const int my_row = (S::kChunks >= 32 ? 0 : lane / S::kChunks) + rg * (kTile / RW), my_chunk = lane % S::kChunks;
  const long long slot_bytes = c.slot_stride * static_cast<int>(sizeof(T));
  const long long my_src = my_row * slot_bytes + my_chunk * 16;
  const unsigned my_dst = swizzled<T, D>(my_row, my_chunk);
  auto look_up = [&] {
    const int key = f.k0 + kTile * kg + f_i * kStep + (c.whole_tiles ? 0 : lane & (kTile - 1));
    page = key < f.k1 ? f_table[c.page_div.div(key)] : 0;
  };
  auto next_item = [&] {  // to the next item in which this key group has a tile
    for (f_any = false; f.find(c, f_u, u1); ) {
      f.pass(f_u);
      f_n = f.tiles_of(kg);
      if (f_n > 0) {
        f_any = true;
        f_i = 0;
        f_head = f.item / f.r.blocks;
        f_table = c.table + static_cast<uint64_t>(f.seq) * c.max_pages;
        look_up();
        break;
      }
    }
  };
  // q of the item, for its first use a whole tile later
  int head = 0, block = 0;
  W w(lane, row0);
  auto begin_q = [&] {
    head = it.item / it.r.blocks;
    block = it.item - head * it.r.blocks;
    // Column n of the score tile is row block * kRows + n of the item: token row / group, query head row % group.
    const int rows = it.r.tokens * static_cast<int>(c.group);
    auto q_row = [&](int n) -> const T * {
      const int row = block * kRows + n;
      if (row >= rows) return nullptr;
      const int t = c.group_div.div(row);
      return static_cast<const T *>(c.q) + static_cast<int64_t>(it.r.t0 + t) * c.q_stride +
             (static_cast<int64_t>(head) * c.group + (row - t * static_cast<int>(c.group))) * D;
    };
    w.load_q(q_row, q_smem, lane, row0);
  };
  long long u = u0;
  bool more = it.find(c, u, u1);
  if (more) begin_q();

  next_item();
  auto fetch = [&] {  // the next half tile: K of a tile, then its V
    if (f_any) {
      const char *base = static_cast<const char *>(f_value ? c.v : c.k);
      const unsigned to = ring + f_slot * S::kHalf;
      if (c.whole_tiles) {  // a tile lies in one page: rows past the end are another request's or stale, and cut out later
        if (!f_value) {
          const int key = f.k0 + kTile * kg + f_i * kStep;
          const int o = key - static_cast<int>(c.page_div.div(key) * c.page_size);
          const bool none = static_cast<uint32_t>(page) >= c.n_pages, seen = key + kTile > f.r.first;
          bad_slots = (bad_slots & ~(1u << f_slot)) | static_cast<unsigned>(none && seen) << f_slot;
          if (none) page = 0;
          row_at = (page * c.page_stride + f_head * c.head_stride) * static_cast<int>(sizeof(T)) + o * slot_bytes;
        }
        const char *src = base + row_at + my_src;
#pragma unroll
        for (int x = 0; x < kAccesses; ++x) {
          const int row = x * 32 / S::kChunks;
          const unsigned dst = to + (my_dst ^ (order<T>(row) << 4)) + row * S::kRowBytes + (S::kChunks > 32 ? (x & 1) * 512 : 0);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src + (S::kChunks > 32 ? (x & 1) * 512 : 0)) : "memory");
          if (S::kChunks <= 32 || (x & 1)) src += kPer * slot_bytes;
        }
      } else {
        if (!f_value) {
          const int key = f.k0 + kTile * kg + f_i * kStep + (lane & (kTile - 1));
          const int o = key - static_cast<int>(c.page_div.div(key) * c.page_size);
          const bool none = static_cast<uint32_t>(page) >= c.n_pages, seen = key >= f.r.first && key < f.k1;
          bad_slots = (bad_slots & ~(1u << f_slot)) | static_cast<unsigned>(none && seen) << f_slot;
          row_at = key < f.k1 && !none
                       ? (page * c.page_stride + f_head * c.head_stride) * static_cast<int>(sizeof(T)) + o * slot_bytes
                       : -1;
        }
#pragma unroll 4
        for (int x = rg * kAccesses; x < (rg + 1) * kAccesses; ++x) {
          const int row = (x * 32 + lane) / S::kChunks, ch = (x * 32 + lane) % S::kChunks;
          const long long off = __shfl_sync(kFull, row_at, row);
          cp_async_16_or_zero(to + swizzled<T, D>(row, ch), base + (off < 0 ? 0 : off) + ch * 16, off >= 0);
        }
      }
      f_slot = f_slot + 1 == kRing ? 0 : f_slot + 1;
      if (f_value) {
        if (++f_i < f_n) look_up();
        else next_item();
      }
      f_value = !f_value;
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int h = 0; h < kRing - 1; ++h) fetch();
  // Before a half tile is used: its copies are there, for every warp of the group, and all of them are done with
  // the one before, whose slot the next copies take.
  auto arrived = [&] {
    cp_async_wait<kRing - 2>();
    if constexpr (RW == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;\n" ::"r"(1 + kg), "n"(32 * RW) : "memory");
    fetch();
  };

  unsigned slot = 0;
  while (more) {
    const Request &r = it.r;
    const int rows = r.tokens * static_cast<int>(c.group);
    // the last key each of this lane's columns sees
    int last[NT][2], token[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = min(block * kRows + row0 + nt * 8 + (lane & 3) * 2 + j, rows - 1);
        token[nt][j] = c.group_div.div(row);
        last[nt][j] = r.len - r.tokens + token[nt][j];
      }
    const int t_first = c.group_div.div(min(block * kRows + row0, rows - 1));
    const int t_last = c.group_div.div(min(block * kRows + row0 + NT * 8, rows) - 1);
    // keys in [all0, all1) are seen by every row of this warp
    const int all1 = min(r.len - r.tokens + t_first + 1, it.k1);
    const int all0 = c.window ? less_window(r.len - r.tokens + t_last + 1, c.window) : 0;
    if (W::kQSmem) __syncthreads();

    // Sums are kept relative to 2^m; m follows the running maximum only when that has grown by more than
    // 2^8, so that the rescaling is rare (a probability is then below 2^8, far from f32's range).  Starting
    // from the lowest finite value, a column that sees nothing keeps zero sums.
    float acc[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.0f;
      m[nt][0] = m[nt][1] = kLowest;
      l[nt][0] = l[nt][1] = 0.0f;
    }

    const bool short_sums = it.k1 - it.k0 <= kShortKeys * KW;
    const int n_tiles = it.tiles_of(kg);
    int key0 = it.k0 + kTile * kg;
    bool bad_page = false;
#pragma unroll 1
    for (int i = 0; i < n_tiles; ++i, key0 += kStep) {
      // scores
      arrived();
      float s[KT][NT][4];
      const bool edge = key0 + kTile > all1 || key0 < all0;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) w.scores(s[kt], ring + slot * S::kHalf + kt * kSub * S::kRowBytes, q_smem);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[kt][nt][j] *= c.scale_log2;
      if (edge) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int key = key0 + kt * kSub + lane / 4 + (j >> 1) * 8, hi = min(last[nt][j & 1], it.k1 - 1);
              const long long lo = c.window ? static_cast<long long>(last[nt][j & 1]) - c.window : -1;
              if (key > hi || key <= lo) s[kt][nt][j] = -INFINITY;
            }
      }
      bad_page |= bad_slots >> slot & 1;
      slot = slot + 1 == kRing ? 0 : slot + 1;
      bool grown = false;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) grown |= s[kt][nt][j] > m[nt][j & 1] + 8.0f;
      if (__any_sync(kFull, grown)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float g[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(s[0][nt][j], s[0][nt][j + 2]);
#pragma unroll
            for (int kt = 1; kt < KT; ++kt) top = fmaxf(top, fmaxf(s[kt][nt][j], s[kt][nt][j + 2]));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 4));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 8));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 16));
            top = fmaxf(top, m[nt][j]);
            g[j] = exp2_fast(m[nt][j] - top);
            m[nt][j] = top;
            l[nt][j] *= g[j];
          }
#pragma unroll
          for (int md = 0; md < D / 16; ++md) {
            acc[md][nt][0] *= g[0];
            acc[md][nt][1] *= g[1];
            acc[md][nt][2] *= g[0];
            acc[md][nt][3] *= g[1];
          }
        }
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            s[kt][nt][j] = exp2_fast(s[kt][nt][j] - m[nt][j]);
            s[kt][nt][j + 2] = exp2_fast(s[kt][nt][j + 2] - m[nt][j]);
            l[nt][j] += s[kt][nt][j] + s[kt][nt][j + 2];
          }
      typename W::P p[KT];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) p[kt].take(s[kt], lane);
      // output
      arrived();
      const unsigned v_tile = ring + slot * S::kHalf;
      slot = slot + 1 == kRing ? 0 : slot + 1;
      // the tile's values, those of keys outside [from, to) as zeros; into the running sums or beside them
      auto weigh = [&](auto direct, auto cut, int from, int to) {
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          float y[NT][4] = {};
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            typename W::V v(w, v_tile + kt * kSub * S::kRowBytes, md);
            if constexpr (cut()) v.keep(from - kt * kSub, to - kt * kSub, lane);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) v.mma(direct() ? acc[md][nt] : y[nt], p[kt], nt);
          }
          if constexpr (!direct()) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[md][nt][j] += y[nt][j];
          }
        }
      };
      if (!edge) {
        if (kKeepsShortSums<T, D, NT> && short_sums) weigh(std::bool_constant<kKeepsShortSums<T, D, NT>>{}, std::false_type{}, 0, 0);
        else weigh(std::false_type{}, std::false_type{}, 0, 0);
        continue;
      }
      // A key that a token does not see must not reach its row even as 0 * v (v may be stale, infinite or NaN).
      // Keys that no token of the warp sees are cut out of V; if tokens see different keys of the tile and a
      // value of those is not finite, each token's columns take a product of their own.
      const int seen0 = c.window ? less_window(r.len - r.tokens + t_first + 1 - key0, c.window) : 0;
      const int seen1 = min(r.len - r.tokens + t_last + 1, it.k1) - key0;
      bool apart = false;
      if (t_first != t_last) {
        unsigned most = 0;
#pragma unroll 4
        for (int md = 0; md < D / 16; ++md) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            typename W::V v(w, v_tile + kt * kSub * S::kRowBytes, md);
            v.keep(seen0 - kt * kSub, seen1 - kt * kSub, lane);
            v.largest(most);
          }
        }
        apart = __any_sync(kFull, !W::V::finite(most));
      }
      if (!apart) {
        constexpr bool kDirect = kKeepsShortSums<T, D, NT> && D != 128;
        if (kDirect && short_sums) weigh(std::bool_constant<kDirect>{}, std::true_type{}, seen0, seen1);
        else weigh(std::false_type{}, std::true_type{}, seen0, seen1);
      } else {
#pragma unroll 1
        for (int t = t_first; t <= t_last; ++t) {
          const int hi = r.len - r.tokens + t + 1 - key0;
          const int lo = c.window ? less_window(hi, c.window) : 0;
#pragma unroll
          for (int md = 0; md < D / 16; ++md) {
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              typename W::V v(w, v_tile + kt * kSub * S::kRowBytes, md);
              v.keep(lo - kt * kSub, min(hi, it.k1 - key0) - kt * kSub, lane);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                v.mma(y, p[kt], nt);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (token[nt][j & 1] == t) acc[md][nt][j] += y[j];
              }
            }
          }
        }
      }
    }

    // Join the key groups.
    bad_page = __any_sync(kFull, bad_page);
    if (lane == 0) s_bad[warp] = bad_page;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float x = l[nt][j];
        x += __shfl_xor_sync(kFull, x, 4);
        x += __shfl_xor_sync(kFull, x, 8);
        x += __shfl_xor_sync(kFull, x, 16);
        if (lane < 4) {
          s_m[warp][nt * 8 + lane * 2 + j] = m[nt][j];
          s_l[warp][nt * 8 + lane * 2 + j] = x;
        }
      }
    const bool whole = it.tile0 == 0 && it.tile1 == r.tiles;
    const int part_slot = 2 * cta + (u == u0 ? 0 : 1);  // an item that goes on from the CTA before is the share's first
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int d0 = 0; d0 < D; d0 += kJoinCols) {
#pragma unroll
        for (int md = 0; md < kJoinCols / 16; ++md)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            join[(warp * 8 + (lane & 3) * 2 + (j & 1)) * kJoinRow + md * 16 + lane / 4 + (j >> 1) * 8] = acc[d0 / 16 + md][nt][j];
        __syncthreads();
        bool poison = false;  // rows over a page that does not exist are NaN
#pragma unroll
        for (int i = 0; i < WARPS; ++i) poison |= s_bad[i] != 0;
        if (poison && tid == 0) report(GDN_DEVICE_BAD_PAGE);
#pragma unroll 1
        for (int x = tid; x < RW * 8 * kJoinCols / 4; x += kThreads) {
          const int row = x / (kJoinCols / 4), d = x % (kJoinCols / 4) * 4;
          const int of = row / 8, in = row % 8, m_row = nt * 8 + in;  // rows of warps of, of + RW, ...
          const int n = of * NT * 8 + m_row, item_row = block * kRows + n;
          if (item_row >= rows) break;
          float top = s_m[of][m_row];
#pragma unroll
          for (int i = 1; i < KW; ++i) top = fmaxf(top, s_m[i * RW + of][m_row]);
          float sum[4] = {}, den = 0.0f;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            const float g = exp2_fast(s_m[i * RW + of][m_row] - top);
            const float4 y = *reinterpret_cast<const float4 *>(join + ((i * RW + of) * 8 + in) * kJoinRow + d);
            sum[0] += g * y.x;
            sum[1] += g * y.y;
            sum[2] += g * y.z;
            sum[3] += g * y.w;
            den += g * s_l[i * RW + of][m_row];
          }
          if (poison) den = NAN;
          if (whole) {
            const float inv = 1.0f / den;
            const int t = c.group_div.div(item_row);
            // a row that sees no key is zero; one whose visible scores are all -inf is 0 / 0
            const bool empty = r.len - r.tokens + t < 0 && !poison;
            T *o = static_cast<T *>(c.out) + static_cast<int64_t>(r.t0 + t) * c.out_stride +
                   (static_cast<int64_t>(head) * c.group + (item_row - t * static_cast<int>(c.group))) * D + d0 + d;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = empty ? 0.0f : sum[e] * inv;
            put4(o, sum, c.out_wide);
          } else {
            const size_t at = static_cast<size_t>(part_slot) * kRows + n;
            *reinterpret_cast<float4 *>(c.part + at * D + d0 + d) = make_float4(sum[0], sum[1], sum[2], sum[3]);
            if (d0 + d == 0) c.part_ml[at] = make_float2(top, den);
          }
        }
        __syncthreads();
      }
    }
    if (!whole && it.tile0 == 0 && tid == 0) {
      const long long end = u + it.units + (r.tiles - it.tile1) - 1;  // the item's last unit
      c.splits[cta] = Split{part_slot, static_cast<int>(((end + 1) * ctas - 1) / total), block * kRows, rows, r.t0,
                            head * static_cast<int>(c.group), r.len - r.tokens};
    }
    it.pass(u);
    more = it.find(c, u, u1);
    if (more) begin_q();
  }
  cp_async_wait<0>();
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
uint64_t rows_of(const gdn_attn_params &p) {
  const uint64_t window = (p.n_tokens + static_cast<uint64_t>(p.n_seqs) - 1) / p.n_seqs;
  return window * (p.n_q_heads / p.n_kv_heads);
}

template <typename T, int D_, int NT_, int RW_, int WARPS_ = 4, int KT_ = 1>
struct Pick {
  using type = T;
  static constexpr int D = D_, NT = NT_, RW = RW_, WARPS = WARPS_, KT = KT_, rows = NT_ * RW_ * 8;
  static constexpr int ctas = kSms * ctas_per_sm<T, D_, NT_, RW_, WARPS_, KT_>();
};

// Calls f with the Pick of the call: the fewest rows per block that hold its
// rows.  A block of 8 costs what the cache's bytes cost; more rows raise the
// work per byte, first on a warp's second tile, then on more warps per ring.
template <typename F>
auto dispatch(const gdn_attn_params &p, F f) {
  const uint64_t rows = rows_of(p);
  auto by_rows = [&](auto t, auto d) {
    using T = decltype(t);
    constexpr int D = d();
    if constexpr (sizeof(T) * D >= 1024) {  // 1 KB per key: no room for more than 8 rows of q beside the rings
      return f(Pick<T, D, 1, 1>{});
    } else if constexpr (D == 256) {  // 16 columns' accumulators and q would not fit a thread's registers
      // 17 to 24 rows take one block of 32 rather than two of 16, which read every key twice (64 requests up to 8192
      // keys, 17 to 24 heads on each of 4: 205 against 302 us; 32 requests, 2 key heads: 65 against 86) -- but where
      // that is an average of windows of different lengths, many requests have 16 rows or less (32 requests, windows
      // of 1 to 4 tokens, 8 heads on each of 2: 67 against 61).
      const bool some_narrow = p.n_tokens % p.n_seqs != 0 && p.n_q_heads / p.n_kv_heads <= 16;
      return rows <= 8                           ? f(Pick<T, D, 1, 1>{})
             : rows <= (some_narrow ? 24u : 16u) ? f(Pick<T, D, 1, 2, 8>{})
                                                 : f(Pick<T, D, 1, 4, 8, 2>{});
    } else if constexpr (sizeof(T) == 4) {
      return rows <= 8 ? f(Pick<T, D, 1, 1>{}) : rows <= 16 ? f(Pick<T, D, 2, 1>{}) : f(Pick<T, D, 2, 2>{});
    } else {
      // at 128 bytes a key, steps of 32 keys halve what a step costs beside its loads (64 requests up to 8192
      // keys, 32/8 heads: 89.1 -> 85.4 us); at 256 bytes they cost registers (81.0 -> 85.4 us)
      return rows <= 8    ? f(Pick<T, D, 1, 1, 4, D == 64 ? 2 : 1>{})
             : rows <= 16 ? f(Pick<T, D, 2, 1>{})
             : rows <= 32 ? f(Pick<T, D, 2, 2, 4, 2>{})
                          : f(Pick<T, D, 2, 4, 4, 2>{});
    }
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
  return dispatch(p, [&](auto pick) {
    using P = decltype(pick);
    return part_floats(P::ctas, P::rows, P::D) * 4 + static_cast<size_t>(2) * P::ctas * P::rows * sizeof(float2) +
           P::ctas * sizeof(Split);
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
  const uintptr_t four = p.dtype == GDN_DTYPE_BF16 ? 8 : 16;
  c.out_wide = reinterpret_cast<uintptr_t>(a.output) % four == 0 && p.out_stride % 4 == 0;
  return dispatch(p, [&](auto pick) {
    using P = decltype(pick);
    using T = typename P::type;
    constexpr int smem = smem_bytes<T, P::D, P::NT, P::RW, P::WARPS, P::KT>();
    c.whole_tiles = p.page_size % (kSub * P::KT) == 0;
    // An item of a few units is not split: the join of its parts would take longer than its keys (16 requests,
    // 16/4 heads of 128, bf16, up to 256 keys: 8.7 split, 7.9 us whole; up to 512: 8.9, 10.8; f32 up to 128 keys: 10.3,
    // 9.0; up to 256: equal).
    const uint64_t seen = static_cast<uint64_t>(p.window) + p.n_tokens;  // keys a window of tokens sees at most
    const uint64_t keys = static_cast<uint64_t>(p.max_pages) * p.page_size;
    c.whole_items = (p.window && seen < keys ? seen : keys) <= (sizeof(T) == 4 ? 128 : 256);
    c.splits = static_cast<Split *>(a.workspace);
    c.part = reinterpret_cast<float *>(c.splits + P::ctas);
    c.part_ml = reinterpret_cast<float2 *>(c.part + part_floats(P::ctas, P::rows, P::D));
    const auto main = gdn_attn_paged_kernel<T, P::D, P::NT, P::RW, P::WARPS, P::KT>;
    cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_in_order(main, dim3(P::ctas), 32 * P::WARPS, smem, stream, c);
    if (e != cudaSuccess || c.whole_items) return e;
    // Few items have many parts each: several warps per row; many have few: a warp per row.
    constexpr int kFewPer = P::rows / 4 < kJoinWarps ? P::rows / 4 : kJoinWarps;
    const bool few = static_cast<uint64_t>(p.n_seqs) * p.n_kv_heads * 4 < P::ctas;
    return launch_in_order(few ? gdn_attn_join_kernel<T, P::D, P::rows, kFewPer> : gdn_attn_join_kernel<T, P::D, P::rows, kJoinWarps>,
                           dim3(P::ctas, P::rows / (few ? kFewPer : kJoinWarps)), 32 * kJoinWarps, 0, stream, c);
  });
}

cudaError_t attn_paged_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
