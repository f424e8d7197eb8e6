// Attention of each request's newest tokens over its 8-bit paged cache
// (gdn_attn_paged_fp8): out = sum_j softmax_j(scale q.k_j) v_j, where an element
// of k_j and v_j is an e4m3 code times the scale of its page and key head.
//
// What bounds it.  Every code is read once and used for group x window rows: 4 to
// 200 flops a byte, so HBM bounds it up to some 16 rows per key head, as it bounds
// the kernel over a bf16 cache, at half the bytes.  The same structure serves (its
// file gives the reasons): a token's rows on the N side of the warp-level matrix
// instruction (S^T = K Q^T, O^T = V^T P^T), shares of a list of units, a ring of
// half tiles per key group that runs on across items.  What differs is how codes
// become operands.
//
// Operands.  e4m3 is a part of f16, so a code is exact there, and the products are
// those of f16 matrix instructions with f32 sums.  q goes in with each row scaled
// by a power of two to below 2^14 (exact for bf16; f32 as two halves), the
// probabilities relative to a maximum such that they lie below 2^15 and lose
// nothing above 2^-35 of the largest.  The contraction of a product may go
// in any order, so the order is that of the memory: a lane takes 16 neighbouring
// bytes of a key for four steps of Q K^T, and 16 neighbouring elements of four
// values for eight steps of P V, whose result then has 16 neighbouring elements in
// each lane.  So shared memory is read 16 bytes at a time, and nothing is
// transposed but bytes of two keys in registers.
//
// Scales.  A key's scale multiplies its scores.  A tile's values are summed as
// codes, times their page's scale over the largest of the tile, and the sums are
// added to the running ones, in f32, times that largest.  Where scales of a tile
// are further apart than 2^8 its pages take products of their own.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "attn_work.cuh"
#include "fp8_common.cuh"

namespace gdn {
namespace {

constexpr float kLargest = 3.402823466e38f;
// A probability is kept times 2^kTopBits, relative to a maximum that may lag by a factor of 2^kLagBits: f16 holds up to
// 2^16, and down to 2^-24.
constexpr float kTopBits = 11.0f, kLagBits = 4.0f;

// c += a (16 x 16) b (16 x 8), f16
__device__ __forceinline__ void mma_f16(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ unsigned f16x2(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const unsigned *>(&h);
}
__device__ __forceinline__ float2 f32x2(unsigned h) { return __half22float2(*reinterpret_cast<const __half2 *>(&h)); }

template <int N>
struct Words {
  unsigned w[N];
};
__device__ __forceinline__ void load_words(Words<4> &x, unsigned addr) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n" : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void load_words(Words<2> &x, unsigned addr) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];\n" : "=r"(x.w[0]), "=r"(x.w[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ float load_f32(unsigned addr) {
  float x;
  asm volatile("ld.shared.f32 %0, [%1];\n" : "=f"(x) : "r"(addr) : "memory");
  return x;
}

// A half tile in shared memory: kTile rows of codes, then, beside K, the scales of its keys and of their values.
template <int D, int KT>
struct Shape8 {
  static constexpr int kTile = kSub * KT;
  static constexpr int kChunks = D / 16;  // 16-byte chunks per row
  static constexpr int kCodes = kTile * D;
  static constexpr int kHalf = kCodes + 2 * kTile * 4;
  static constexpr int kSteps = D / 16;   // matrix steps of Q K^T
  static constexpr int kBytes = D >= 128 ? 16 : 8;  // neighbouring elements that a lane takes of a value at once
  static constexpr int kPieces = D / (8 * kBytes);  // such pieces of a row
};

// Where chunk c of row r lies.  K: lanes read chunks 0-3 or 4-7 of rows r and r + 1 at once; rows of 128 bytes and
// more exchange the two in odd rows.  V: lanes read two neighbouring chunks (64 elements: one) of rows r, r + 2,
// r + 4 and r + 6 at once; rows of 64 bytes are put in such an order that these follow one another.  Either way eight
// lanes' 16 bytes (16 lanes' 8) fall on different banks.  The chunk's place is linear over XOR in the row's low bits.
template <int D>
__device__ __forceinline__ constexpr int k_order(int r) {
  return D >= 128 ? (r & 1) << 2 : 0;
}
template <int D>
__device__ __forceinline__ constexpr int v_order(int r) {
  return D >= 128 ? (r >> 1 & 3) << 1 : (r >> 2 & 1) << 1;
}
template <int D>
__device__ __forceinline__ constexpr int v_row(int r) {
  return D >= 128 ? r : (r & ~7) + (r >> 1 & 3) + (r & 1) * 4;
}
template <int D>
__device__ __forceinline__ constexpr int k_place(int r, int c) {
  return r * D + ((c ^ k_order<D>(r)) << 4);
}
template <int D>
__device__ __forceinline__ constexpr int v_place(int r, int c) {
  return v_row<D>(r) * D + ((c ^ v_order<D>(r)) << 4);
}

// What a warp has of q and does with a tile.  HALVES: f16 halves of q and of the probabilities (bf16 1, f32 2).
template <typename T, int D, int NT, int KT>
struct Warp8 {
  using S = Shape8<D, KT>;
  static constexpr int kHalves = sizeof(T) == 4 ? 2 : 1;
  unsigned q[S::kSteps][NT][kHalves][2];
  float by[NT][2];  // what takes the column's sums of codes to scores in the log2 domain
  unsigned k_at, v_at[4];  // this lane's offsets: of row lane / 4; of values 2 t, 2 t + 1, 2 t + 8, 2 t + 9, t = lane % 4

  __device__ __forceinline__ explicit Warp8(int lane) {
    k_at = k_place<D>(lane / 4, lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (lane & 3) * 2 + (i & 1) + (i >> 1) * 8;
      v_at[i] = S::kBytes == 16 ? v_place<D>(r, lane / 4) : v_place<D>(r, lane / 8) + (lane / 4 & 1) * 8;
    }
  }

  // row(n): q's row of column n of the block, or nullptr; this warp's begin at row0
  template <typename F>
  __device__ __forceinline__ void load_q(F row, int lane, int row0, float scale_log2) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const T *p = row(row0 + nt * 8 + lane / 4);
      // step ks of 64-element group ks / 4: elements (lane % 4) * 16 + ks % 4 * 4 .. + 4 of the group
      float x[S::kSteps][4], top = 0.0f;
#pragma unroll
      for (int ks = 0; ks < S::kSteps; ++ks) {
        const T *e = p + (ks >> 2) * 64 + (lane & 3) * 16 + (ks & 3) * 4;
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const unsigned u = p ? reinterpret_cast<const unsigned *>(e)[b] : 0u;
            x[ks][2 * b] = __uint_as_float(u << 16);
            x[ks][2 * b + 1] = __uint_as_float(u & 0xffff0000u);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[ks][i] = p ? e[i] : 0.0f;
        }
      }
#pragma unroll
      for (int ks = 0; ks < S::kSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fabsf(x[ks][i]) <= kLargest ? fmaxf(top, fabsf(x[ks][i])) : top;
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      // the row's largest to [2^13, 2^14)
      const int up = top > 0.0f ? min(13 + 127 - (__float_as_int(top) >> 23), 126) : 0;
      const float f = __int_as_float((up + 127) << 23), back = __int_as_float((127 - up) << 23) * scale_log2;
#pragma unroll
      for (int j = 0; j < 2; ++j) by[nt][j] = __shfl_sync(kFull, back, ((lane & 3) * 2 + j) * 4);
#pragma unroll
      for (int ks = 0; ks < S::kSteps; ++ks)
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float u = x[ks][2 * b] * f, v = x[ks][2 * b + 1] * f;
          q[ks][nt][0][b] = f16x2(u, v);
          if constexpr (kHalves == 2) {
            const float2 h = f32x2(q[ks][nt][0][b]);
            q[ks][nt][1][b] = f16x2(u - h.x, v - h.y);
          }
        }
    }
  }

  // s = K Q^T of 16 keys, as sums of codes
  __device__ __forceinline__ void scores(float (&s)[NT][4], unsigned k_tile) const {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.0f;
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      Words<4> lo, hi;
      const unsigned at = k_tile + (k_at ^ ((g & 1) << 6)) + (g >> 1) * 128;
      load_words(lo, at);
      load_words(hi, at + 8 * D);
      float t[NT][4];
      if constexpr (kHalves == 2) {
        // the tensor cores cut the low bits of a running sum: f32's are taken over 64 elements, and added outside
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) t[nt][0] = t[nt][1] = t[nt][2] = t[nt][3] = 0.0f;
      }
      unsigned a[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i][0] = codes_f16x2(lo.w[i], 0);
        a[i][1] = codes_f16x2(hi.w[i], 0);
        a[i][2] = codes_f16x2(lo.w[i], 2);
        a[i][3] = codes_f16x2(hi.w[i], 2);
      }
#pragma unroll
      for (int h = kHalves - 1; h >= 0; --h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(kHalves == 2 ? t[nt] : s[nt], a[i], q[g * 4 + i][nt][h][0], q[g * 4 + i][nt][h][1]);
      if constexpr (kHalves == 2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[nt][j] += t[nt][j];
      }
    }
  }

  // The B fragments of P^T from the score tile's layout.
  struct P {
    unsigned b[NT][kHalves][2];
    __device__ __forceinline__ void take(const float (&p)[NT][4]) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float x = p[nt][2 * i], y = p[nt][2 * i + 1];
          const unsigned h = f16x2(x, y);
          b[nt][0][i] = movmatrix_trans(h);
          if constexpr (kHalves == 2) {
            const float2 z = f32x2(h);
            b[nt][1][i] = movmatrix_trans(f16x2(x - z.x, y - z.y));
          }
        }
    }
  };

  // This lane's part of 16 values: kBytes neighbouring elements of four keys.
  struct V {
    Words<S::kBytes / 4> r[4];
    __device__ __forceinline__ void load(const Warp8 &w, unsigned v_tile, int piece) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words(r[i], v_tile + w.v_at[i] + piece * 128);
    }
    // keys outside [k0, k1) as zeros
    __device__ __forceinline__ void keep(int k0, int k1, int lane) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = (lane & 3) * 2 + (i & 1) + (i >> 1) * 8;
        if (key < k0 || key >= k1)
#pragma unroll
          for (int x = 0; x < S::kBytes / 4; ++x) r[i].w[x] = 0u;
      }
    }
    __device__ __forceinline__ bool has_nan() const {
      unsigned m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < S::kBytes / 4; ++x) m |= (r[i].w[x] & 0x7f7f7f7fu) + 0x01010101u;
      return (m & 0x80808080u) != 0;
    }
    // V^T of elements 2 m and 2 m + 1 of the piece (rows lane / 4 and lane / 4 + 8 of the fragment)
    __device__ __forceinline__ void fragment(unsigned (&a)[4], int m) const {
      const unsigned x = __byte_perm(r[0].w[m >> 1], r[1].w[m >> 1], m & 1 ? 0x7362 : 0x5140);
      const unsigned y = __byte_perm(r[2].w[m >> 1], r[3].w[m >> 1], m & 1 ? 0x7362 : 0x5140);
      a[0] = codes_f16x2(x, 0);
      a[1] = codes_f16x2(x, 2);
      a[2] = codes_f16x2(y, 0);
      a[3] = codes_f16x2(y, 2);
    }
  };
  // y += V^T P^T
  static __device__ __forceinline__ void weigh(float (&y)[4], const unsigned (&a)[4], const P &p, int nt) {
#pragma unroll
    for (int h = kHalves - 1; h >= 0; --h) mma_f16(y, a, p.b[nt][h][0], p.b[nt][h][1]);
  }
};

// The join of a CTA's warps goes through shared memory in pieces of 8 rows x join_cols.
template <int D>
constexpr int join_cols() {
  return D < 256 ? D : 128;
}
template <int D, int WARPS>
constexpr int join_bytes() {
  return WARPS * 8 * (join_cols<D>() + 4) * 4;
}

// A variant: NT 8-row tiles of a warp, RW warps that share a ring, each with rows of its own, WARPS of a CTA, KT matrix
// tiles of 16 keys in a step, CTAS on an SM, SLOTS half tiles in a CTA's rings together.
template <typename T_, int D_, int NT_, int RW_, int WARPS_, int KT_, int CTAS_, int SLOTS_>
struct Pick8 {
  using T = T_;
  static constexpr int D = D_, NT = NT_, RW = RW_, WARPS = WARPS_, KT = KT_, CTAS = CTAS_, SLOTS = SLOTS_;
  static constexpr int rows = NT * RW * 8, ctas = kSms * CTAS;
  static constexpr int smem = SLOTS * Shape8<D, KT>::kHalf + join_bytes<D, WARPS>();
  static_assert((smem + 1024 + 700) * CTAS <= 228 * 1024, "the CTAs fit an SM's shared memory");
};

template <typename P>
__global__ void __launch_bounds__(32 * P::WARPS, P::CTAS) gdn_attn_fp8_kernel(const __grid_constant__ Call c) {
  using T = typename P::T;
  constexpr int D = P::D, NT = P::NT, RW = P::RW, WARPS = P::WARPS, KT = P::KT;
  using S = Shape8<D, KT>;
  using W = Warp8<T, D, NT, KT>;
  constexpr int kTile = S::kTile;
  constexpr int kJoinCols = join_cols<D>(), kJoinRow = kJoinCols + 4;
  constexpr int kRows = P::rows;       // rows of a block
  constexpr int KW = WARPS / RW;       // key groups
  constexpr int kStep = kTile * KW;    // keys from a group's tile to its next
  constexpr int kRing = P::SLOTS / KW;
  static_assert(kRing >= 3 && kRing <= 32, "a bit per slot");
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[WARPS], s_offset;
  __shared__ uint32_t s_seq;
  __shared__ float s_m[WARPS][NT * 8], s_l[WARPS][NT * 8];
  __shared__ int s_bad[WARPS];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int kg = warp / RW, rg = warp % RW, row0 = rg * NT * 8;  // key group; rows of the block
  const unsigned ring = smem_u32(smem) + kg * kRing * S::kHalf;
  float *join = reinterpret_cast<float *>(smem + P::SLOTS * S::kHalf);

  begin_in_order();
  const Share sh = take_share<kRows, WARPS>(c, s_scan, s_seq, s_offset);
  if (sh.cta >= sh.ctas) return;
  const int cta = sh.cta, ctas = sh.ctas;
  const long long total = sh.total, u0 = sh.u0, u1 = sh.u1;

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
  unsigned bad_slots = 0;  // bit i: a page of the K tile in slot i of the ring is none of the cache's, and not wholly
                           // before the window: pages that the window has left may be given back
  // the next tile's pages, looked up a tile ahead: of its 16-key parts, or of this lane's row
  constexpr int kPer = 32 / S::kChunks;                    // rows one access of the warp covers
  constexpr int kAccesses = kTile * S::kChunks / 32 / RW;  // of this warp for a half tile
  static_assert(kAccesses >= 1, "every warp of a key group has a part of a half tile");
  int page[KT];
  long long row_at[KT];  // byte offset of the part's first row (of this lane's row; -1: zeros) in the caches
  const int my_row = lane / S::kChunks + rg * (kTile / RW), my_chunk = lane % S::kChunks;
  const long long my_src = (my_row & (kSub - 1)) * c.slot_stride + my_chunk * 16;
  const unsigned my_k = k_place<D>(my_row, my_chunk), my_v = v_place<D>(my_row, my_chunk);
  auto look_up = [&] {
    const int key = f.k0 + kTile * kg + f_i * kStep;
    if (c.whole_tiles) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) page[kt] = key + kt * kSub < f.k1 ? f_table[c.page_div.div(key + kt * kSub)] : 0;
    } else {
      const int mine = key + (lane & (kTile - 1));
      page[0] = mine < f.k1 ? f_table[c.page_div.div(mine)] : 0;
    }
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
  int head = 0, block = 0;
  W w(lane);
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
    w.load_q(q_row, lane, row0, c.scale_log2);
  };
  long long u = u0;
  bool more = it.find(c, u, u1);

  next_item();
  auto fetch = [&] {  // the next half tile: K of a tile and both its scales, then its V
    if (f_any) {
      const char *base = static_cast<const char *>(f_value ? c.v : c.k);
      const unsigned to = ring + f_slot * S::kHalf;
      if (!f_value) {
        const int key = f.k0 + kTile * kg + f_i * kStep;
        bool gone = false;
        uint32_t of_scale = 0;  // the page of this lane's key
        if (c.whole_tiles) {  // 16 keys lie in one page: rows past the end are another request's or stale, and cut out later
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            const int k = key + kt * kSub;
            const int o = k - static_cast<int>(c.page_div.div(k) * c.page_size);
            const bool none = static_cast<uint32_t>(page[kt]) >= c.n_pages;
            gone |= none && k + kSub > f.r.first;
            if (none) page[kt] = 0;
            row_at[kt] = page[kt] * c.page_stride + f_head * c.head_stride + o * c.slot_stride;
            if (lane / kSub == kt) of_scale = page[kt];
          }
        } else {
          const int k = key + (lane & (kTile - 1));
          const int o = k - static_cast<int>(c.page_div.div(k) * c.page_size);
          const bool none = static_cast<uint32_t>(page[0]) >= c.n_pages;
          gone = none && k >= f.r.first && k < f.k1;
          row_at[0] = k < f.k1 && !none ? page[0] * c.page_stride + f_head * c.head_stride + o * c.slot_stride : -1;
          of_scale = none ? 0 : page[0];
        }
        bad_slots = (bad_slots & ~(1u << f_slot)) | static_cast<unsigned>(gone) << f_slot;
        if (rg == 0 && lane < kTile) {
          const uint64_t at = static_cast<uint64_t>(of_scale) * c.n_kv + f_head;
          const unsigned dst = to + S::kCodes + lane * 4;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(c.k_scale + at) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst + kTile * 4), "l"(c.v_scale + at) : "memory");
        }
      }
      const unsigned mine = f_value ? my_v : my_k;
      if (c.whole_tiles) {
#pragma unroll
        for (int x = 0; x < kAccesses; ++x) {
          const int row = x * kPer;  // behind my_row
          const long long at = KT == 1 ? row_at[0] : RW == 1 ? row_at[row / kSub] : my_row + row < kSub ? row_at[0] : row_at[KT - 1];
          const unsigned dst = to + (mine ^ ((f_value ? v_order<D>(row) : k_order<D>(row)) << 4)) + row * D;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(base + at + my_src + (row & (kSub - 1)) * c.slot_stride)
                       : "memory");
        }
      } else {
#pragma unroll
        for (int x = 0; x < kAccesses; ++x) {
          const int row = x * kPer;
          const unsigned dst = to + (mine ^ ((f_value ? v_order<D>(row) : k_order<D>(row)) << 4)) + row * D;
          const long long off = __shfl_sync(kFull, row_at[0], my_row + row);
          cp_async_16_or_zero(dst, base + (off < 0 ? 0 : off) + my_chunk * 16, off >= 0);
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
  if (more) begin_q();
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

    // Sums are kept relative to 2^m; m is 2^kTopBits below the running maximum, which it follows only when that has
    // grown by more than 2^kLagBits, so that the rescaling is rare.  Starting from the lowest finite value, a column
    // that sees nothing keeps zero sums.
    float acc[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.0f;
      m[nt][0] = m[nt][1] = kLowest;
      l[nt][0] = l[nt][1] = 0.0f;
    }

    const int n_tiles = it.tiles_of(kg);
    int key0 = it.k0 + kTile * kg;
    bool bad_page = false;
#pragma unroll 1
    for (int i = 0; i < n_tiles; ++i, key0 += kStep) {
      // scores
      arrived();
      const unsigned k_tile = ring + slot * S::kHalf;
      float s[KT][NT][4];
      const bool edge = key0 + kTile > all1 || key0 < all0;
      // keys that a row of this warp sees, of the tile
      const int seen0 = edge && c.window ? less_window(r.len - r.tokens + t_first + 1 - key0, c.window) : 0;
      const int seen1 = edge ? min(r.len - r.tokens + t_last + 1, it.k1) - key0 : kTile;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) w.scores(s[kt], k_tile + kt * kSub * D);
      float vs[KT][2];  // the scales of this lane's keys' values
      unsigned most = 0u, least = 0xffffffffu;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int key = kt * kSub + h * 8 + lane / 4;
          const float ks = load_f32(k_tile + S::kCodes + key * 4);
          vs[kt][h] = load_f32(k_tile + S::kCodes + (kTile + key) * 4);
          if (key >= seen0 && key < seen1) {
            most = max(most, __float_as_uint(vs[kt][h]));
            least = min(least, __float_as_uint(vs[kt][h]));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) s[kt][nt][2 * h + j] = s[kt][nt][2 * h + j] * w.by[nt][j] * ks;
        }
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
          for (int j = 0; j < 4; ++j) grown |= s[kt][nt][j] > m[nt][j & 1] + (kTopBits + kLagBits);
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
            top = fmaxf(top - kTopBits, m[nt][j]);
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
      // The values' scales: one, or near one another and positive, or not (then `apart`).
      most = __reduce_max_sync(kFull, most);
      least = __reduce_min_sync(kFull, least);
      const float ref = __uint_as_float(most);
      bool apart = !(most < 0x7f800000u && __uint_as_float(least) * 256.0f >= ref) && most != 0u;
      if (most != least && !apart) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float by = most ? vs[kt][h] / ref : 0.0f;  // a key that no row sees has the probability 0
            const bool use = most && by <= 1.0f;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) s[kt][nt][2 * h + j] = use ? s[kt][nt][2 * h + j] * by : 0.0f;
          }
      }
      typename W::P p[KT];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) p[kt].take(s[kt]);
      // output
      arrived();
      const unsigned v_tile = ring + slot * S::kHalf;
      slot = slot + 1 == kRing ? 0 : slot + 1;
      // the tile's values, with CUT those of keys that no row sees as zeros
      auto weigh = [&](auto cut) {
#pragma unroll
        for (int x = 0; x < S::kPieces; ++x) {
          typename W::V v[KT];
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            v[kt].load(w, v_tile + kt * kSub * D, x);
            if constexpr (cut()) v[kt].keep(seen0 - kt * kSub, seen1 - kt * kSub, lane);
          }
#pragma unroll
          for (int md = 0; md < S::kBytes / 2; ++md) {
            float y[NT][4] = {};
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              unsigned a[4];
              v[kt].fragment(a, md);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) W::weigh(y[nt], a, p[kt], nt);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[x * (S::kBytes / 2) + md][nt][j] += ref * y[nt][j];
          }
        }
      };
      if (!edge && !apart) {
        weigh(std::false_type{});
        continue;
      }
      // A key that a token does not see must not reach its row even as 0 * v (v may be stale or NaN).  Keys that no
      // token of the warp sees are cut out of V; if tokens see different keys of the tile and one of those is NaN, each
      // token's columns take products of their own.
      const bool folded = !apart;
      if (folded && t_first != t_last) {
        bool nan = false;
#pragma unroll 1
        for (int x = 0; x < S::kPieces * KT; ++x) {
          typename W::V v;
          v.load(w, v_tile + x % KT * kSub * D, x / KT);
          v.keep(seen0 - x % KT * kSub, seen1 - x % KT * kSub, lane);
          nan |= v.has_nan();
        }
        apart = __any_sync(kFull, nan);
      }
      if (!apart) {
        weigh(std::true_type{});
        continue;
      }
      // Token by token and, where the scales are not in P, page by page.
#pragma unroll 1
      for (int t = t_first; t <= t_last; ++t) {
        const int hi = min(r.len - r.tokens + t + 1, it.k1) - key0;
        int from = c.window ? max(0, less_window(r.len - r.tokens + t + 1 - key0, c.window)) : 0;
        while (from < min(hi, kTile)) {
          int to = min(min(hi, kTile), (from / kSub + 1) * kSub);
          float by = ref;
          if (!folded) {
            const int key = key0 + from;
            to = min(to, from + static_cast<int>(c.page_size) - (key - static_cast<int>(c.page_div.div(key) * c.page_size)));
            by = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float x = __shfl_sync(kFull, vs[kt][h], from % 8 * 4);
                if (from / 8 == kt * 2 + h) by = x;
              }
          }
          const int kt0 = from / kSub;
          typename W::P pk = p[0];
          if (KT > 1 && kt0 > 0) pk = p[KT - 1];
#pragma unroll
          for (int x = 0; x < S::kPieces; ++x) {
            typename W::V v;
            v.load(w, v_tile + kt0 * kSub * D, x);
            v.keep(from - kt0 * kSub, to - kt0 * kSub, lane);
#pragma unroll
            for (int md = 0; md < S::kBytes / 2; ++md) {
              unsigned a[4];
              v.fragment(a, md);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                W::weigh(y, a, pk, nt);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (token[nt][j & 1] == t) acc[x * (S::kBytes / 2) + md][nt][j] += by * y[j];
              }
            }
          }
          from = to;
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
        for (int md = 0; md < kJoinCols / 16; md += 2)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float (&a)[4] = acc[d0 / 16 + md][nt], (&b)[4] = acc[d0 / 16 + md + 1][nt];
            *reinterpret_cast<float4 *>(join + (warp * 8 + (lane & 3) * 2 + j) * kJoinRow + lane / 4 * S::kBytes + md * 2) =
                make_float4(a[j], a[2 + j], b[j], b[2 + j]);
          }
        __syncthreads();
        put_rows<T, D, NT, RW, WARPS, kJoinCols>(c, End{&r, rows, head, block, whole, part_slot}, join, s_m, s_l, s_bad, nt, d0);
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

// ------------------------------------------------------------ host

// Calls f with the variant of the call: the fewest rows per block that hold the rows of its requests.
template <typename F>
auto dispatch(const gdn_attn_params &p, F f) {
  const uint64_t rows = rows_of(p);
  auto by_dim = [&](auto t) {
    using T = decltype(t);
    if (p.head_dim == 64)
      return rows <= 8 ? f(Pick8<T, 64, 1, 1, 4, 2, 3, 24>{}) : rows <= 16 ? f(Pick8<T, 64, 2, 1, 4, 2, 3, 24>{}) : f(Pick8<T, 64, 2, 2, 4, 2, 3, 24>{});
    if (p.head_dim == 128)
      return rows <= 8    ? f(Pick8<T, 128, 1, 1, 4, 2, 2, 20>{})
             : rows <= 16 ? f(Pick8<T, 128, 2, 1, 4, 2, 2, 20>{})
                          : f(Pick8<T, 128, 2, 2, 4, 2, 2, 20>{});
    return rows <= 8    ? f(Pick8<T, 256, 1, 1, 4, 1, 2, 20>{})
           : rows <= 16 ? f(Pick8<T, 256, 1, 2, 8, 1, 1, 24>{})
                        : f(Pick8<T, 256, 1, 4, 8, 2, 1, 16>{});
  };
  return p.dtype == GDN_DTYPE_BF16 ? by_dim(__nv_bfloat16{}) : by_dim(float{});
}

}  // namespace

size_t attn_fp8_workspace_bytes(const gdn_attn_params &p) {
  return dispatch(p, [&](auto pick) {
    using P = decltype(pick);
    return part_floats(P::ctas, P::rows, P::D) * 4 + static_cast<size_t>(2) * P::ctas * P::rows * sizeof(float2) +
           P::ctas * sizeof(Split);
  });
}

cudaError_t launch_attn_paged_fp8(const AttnFp8Args &a, cudaStream_t stream) {
  const gdn_attn_params &p = a.p;
  Call c = call_of(p, a.q, a.k_cache, a.v_cache, a.block_table, a.kv_lens, a.token_start, a.output);
  c.k_scale = a.k_scale;
  c.v_scale = a.v_scale;
  return dispatch(p, [&](auto pick) {
    using P = decltype(pick);
    using T = typename P::T;
    c.whole_tiles = p.page_size % kSub == 0;
    const uint64_t seen = static_cast<uint64_t>(p.window) + p.n_tokens;  // keys a window of tokens sees at most
    const uint64_t keys = static_cast<uint64_t>(p.max_pages) * p.page_size;
    c.whole_items = (p.window && seen < keys ? seen : keys) <= 256;
    c.splits = static_cast<Split *>(a.workspace);
    c.part = reinterpret_cast<float *>(c.splits + P::ctas);
    c.part_ml = reinterpret_cast<float2 *>(c.part + part_floats(P::ctas, P::rows, P::D));
    const auto main = gdn_attn_fp8_kernel<P>;
    cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, P::smem);
    if (e != cudaSuccess) return e;
    e = launch_in_order(main, dim3(P::ctas), 32 * P::WARPS, P::smem, stream, c);
    if (e != cudaSuccess || c.whole_items) return e;
    return launch_join<T, P::D, P::rows>(c, P::ctas, static_cast<uint64_t>(p.n_seqs) * p.n_kv_heads * 4 < P::ctas, stream);
  });
}

cudaError_t attn_fp8_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
