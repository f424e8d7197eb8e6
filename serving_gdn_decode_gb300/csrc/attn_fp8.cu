// Attention of each request's newest tokens over its 8-bit paged cache
// (gdn_attn_paged_fp8): out = sum_j softmax_j(scale q.k_j) v_j, where an element
// of k_j and v_j is an e4m3 code times the scale of its page and key head.
//
// What bounds it.  Every code is read once and used for group x window rows: 4 to
// 200 flops a byte.  HBM bounds 1 to 8 rows per key head; past that the warp-level
// instructions do.  As in the kernel over a cache of f32 or bf16 (attn_paged.cu), a
// token's rows are on the N side of the matrix instruction (S^T = K Q^T, O^T = V^T
// P^T), and the CTAs take shares of a list of units.  What differs is how codes
// become operands, and how they come.
//
// Operands.  e4m3 is a part of f16, so a code is exact there (one instruction for
// two), and the products are those of f16 matrix instructions with f32 sums.  q goes
// in with each row scaled by a power of two to below 2^14 (exact for bf16 down to
// 2^-31 of the row's largest; f32 as two halves), the probabilities relative to a
// maximum such that they lie below 2^15.  f16 rounds one by 2^-11 of itself at most,
// to either side, an eighth of what the result's rounding to bf16 takes; for f32 it is
// two halves, 2^-22.  (Two halves for bf16 too, good to 2^-22, would take 59.6 us in place
// of 52.2 for 64 requests, 182 in place of 168 for 256 and 113 in place of 67 for windows.)
// Either way it loses up to 2^-25 where it is small, 2^-36 of the largest; see Scales.  The contraction
// of a product may go in any order, so the order is that of the memory: a lane takes
// 16 neighbouring bytes of a key for four steps of Q K^T, and 16 neighbouring elements
// of four values for eight steps of P V, whose result then has 16 neighbouring elements
// in each lane.  So shared memory is read 16 bytes at a time without bank conflicts,
// and nothing is transposed but bytes of two keys in registers.
//
// Scales.  A key's scale multiplies its scores.  A tile's values are summed as
// codes, times their page's scale over the largest of the tile, and the sums are
// added to the running ones, in f32, times that largest.  Where scales of a tile
// are further apart than 2^8 its pages take products of their own.  What f16 cuts off
// a small probability would show where its value's scale is far above that of the key
// with the maximum: once a tile's largest scale is more than 2^5 (f32: 2) times the
// smallest before it, each column of its probabilities is first lifted to the top of
// f16's range by a power of two.  So a probability times its scale is good to 2^-11 (2^-22)
// of itself or 2^-31 (2^-35) of the row's largest such product.  (64 requests whose value
// scales differ by up to 2^6: 55.0 us in place of 51.5; windows: 72 in place of 61.7.  A test
// of each column's probabilities in place of the scales took 66 for the windows whatever they held.)
//
// Feeding.  Some warps of a CTA do nothing but fill a ring of tiles, by tensor copies
// of boxes of a page's rows, across items; the others take its tiles in turn.  So these
// have neither the copies' instructions nor their registers, hold no request (an item
// comes to them as a job in shared memory), and more of them fit an SM: 12 warps of
// 168 registers.  With the copies in every warp, a ring for each (8 warps of 240
// registers): 64 requests of up to 4096 keys, 32/8 heads of 128, bf16: 68 us, now 51.5;
// 256 requests, 48/8 heads: 214, now 168.  A feeding warp needs 600 to 900 clocks for a
// tile, all latency, an SM's share of HBM one in 360: hence two in each of two CTAs.
//
// Waits.  Every wait on a barrier is bounded.  Where one runs out the warp ends there and
// tells the others, nothing is put from then on that would need it, parts that the join
// looks for are NaN, and the feeding warps end only after their copies have landed.
//
// Measured on a GB300, back to back over three sets of buffers, as shares of the
// measured copy bandwidth (6767 GB/s): 256 requests as above 168 us, 0.93; 64: 51.5 us,
// 0.78; one request of 400 009 keys, 32/4 heads of 128: 75.2 us, 0.81 (in between 0.97:
// 5 us until the first tile -- lengths, pages, tile and q are dependent reads -- and 7 for
// the join); 32 requests, windows of 1 to 4, 16/2 heads of 256: 61.7 us, 0.31; f32, 24
// requests with a window of 1000 keys, 16/16 heads of 64: 19.8 us; pages of 24, 24/8
// heads of 64: 20.1 us.  32 requests up to 4096 keys, 8 key heads of 128, by rows per key
// head: 8: 35.4 us, 16: 48.8, 32: 70.7 (over a bf16 cache 55.9, 60.5, 82.7).  One request
// of 1021 keys, 16/2 heads of 256: 11.4 us, over a bf16 cache 8.8; 4096 new tokens of
// one request, 32/8 heads of 128: 3.68 ms, over a bf16 cache 3.45.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cmath>
#include <mutex>
#include <numeric>
#include <type_traits>

namespace gdn {
namespace {
constexpr int kItemUnits = 4;  // what an item's begin and end cost beside its keys, in units
}
}  // namespace gdn

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
// c = a b
__device__ __forceinline__ void mma_f16_first(float (&c)[4], const unsigned (&a)[4], unsigned b0, unsigned b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
               : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
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


__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// Arrives once this thread's copies so far are done.
__device__ __forceinline__ void mbar_arrive_after_copies(unsigned bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bar) : "memory");
}
// True for one lane of the warp.
__device__ __forceinline__ bool elected() {
  unsigned one;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}
constexpr unsigned kWaitClocks = 2000000000;  // about a second
constexpr unsigned kSleepClocks = 1 << 22;    // shorter limits are waited for awake: a warp may sleep for a good part of this

// Whether the phase has ended, for the whole warp alike; SLEEP: or does within a time that the hardware sets.
template <bool SLEEP>
__device__ __forceinline__ bool mbar_ended(unsigned bar, unsigned phase) {
  unsigned done;
  if constexpr (SLEEP)
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(bar), "r"(phase) : "memory");
  else
    asm volatile("{\n.reg .pred p;\nmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(done) : "r"(bar), "r"(phase) : "memory");
  return __all_sync(kFull, done != 0u);
}
// Whether it ends within `clocks` from now, and before *failed, for the whole warp alike; looked at once more after that.
__device__ __forceinline__ bool mbar_wait_on(unsigned bar, unsigned phase, unsigned clocks, const volatile int *failed) {
  const unsigned t0 = static_cast<unsigned>(clock());
  bool done, late;
  do {
    late = __any_sync(kFull, static_cast<unsigned>(clock()) - t0 > clocks || (failed && *failed));
    done = clocks > kSleepClocks ? mbar_ended<true>(bar, phase) : mbar_ended<false>(bar, phase);
  } while (!done && !late);
  return done;
}
__device__ __noinline__ bool mbar_wait_on_call(unsigned bar, unsigned phase, unsigned clocks, const volatile int *failed) {
  return mbar_wait_on(bar, phase, clocks, failed);
}
// CALL: the wait proper is a function of its own.  Shapes of two row tiles, whose loops are long, gain by it (32 requests up to
// 4096 keys, bf16, 16 rows per key head of 64 / 128 / 256: 35.6 / 48.8 / 58.7 us, else 37.0 / 51.4 / 63.1), those of one lose
// (8 rows: 28.8 / 35.3 / 40.1, else 27.7 / 35.3 / 39.2).
template <bool CALL>
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned phase, unsigned clocks, const volatile int *failed) {
  if (mbar_ended<false>(bar, phase)) return true;
  if constexpr (CALL) return mbar_wait_on_call(bar, phase, clocks, failed);
  else return mbar_wait_on(bar, phase, clocks, failed);
}

// Arrives, and expects `bytes` of copies that report to the barrier themselves.
__device__ __forceinline__ void mbar_expect(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}
// A box of a cache, at element e and place o of key head h and page p, by one thread.
__device__ __forceinline__ void copy_box(unsigned dst, const CUtensorMap *map, int e, int o, int h, int p, unsigned bar) {
  asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];\n"
               ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(e), "r"(o), "r"(h), "r"(p), "r"(bar) : "memory");
}

// A stage of the ring: a tile's rows of K, then of V, in parts of 128 elements (64, where a head has no more).
template <int D, int KT>
struct Shape8 {
  static constexpr int kTile = kSub * KT;
  static constexpr int kRow = D < 128 ? D : 128;  // of a part
  static constexpr int kParts = D / kRow;
  static constexpr int kPart = kTile * kRow;
  static constexpr int kCodes = kTile * D;  // of K, of V
  static constexpr int kStage = 2 * kCodes;
  static constexpr int kSteps = D / 16;   // matrix steps of Q K^T
  static constexpr int kBytes = D >= 128 ? 16 : 8;  // neighbouring elements that a lane takes of a value at once
};

// Where chunk c of row r lies: as the tensor copies' swizzle of 128 (64) bytes has it.  Linear over XOR in r's low bits.
template <int D>
__device__ __forceinline__ constexpr int order(int r) {
  return D >= 128 ? r & 7 : r >> 1 & 3;
}
template <int D, int KT>
__device__ __forceinline__ constexpr int place(int r, int c) {
  using S = Shape8<D, KT>;
  return c / 8 * S::kPart + r * S::kRow + (((c & 7) ^ order<D>(r)) << 4);
}
// The key of a score tile's row g of 8.  Lanes read chunks 0-3 or 4-7 of K of two neighbouring rows g at once, and one
// or two neighbouring chunks of V of rows g, g + 2, g + 4 and g + 6: with these keys, all of either on different banks.
template <int D>
__device__ __forceinline__ constexpr int key_of(int g) {
  return D >= 128 ? g ^ (g & 1) << 2 : ((g >> 1 & 1) | (g & 4)) ^ (g & 1) * 3;
}
template <int D>
__device__ __forceinline__ constexpr int row_of(int key) {  // the reverse
  return D >= 128 ? key ^ (key & 1) << 2 : (key >> 1 & 1) | ((key ^ key >> 1) & 1) << 1 | (key & 4);
}

// What a warp has of q and does with a tile.  Q_SMEM: its fragments of q are in shared memory, not in registers.
template <typename T, int D, int NT, int KT, bool Q_SMEM>
struct Warp8 {
  using S = Shape8<D, KT>;
  static constexpr int kHalves = sizeof(T) == 4 ? 2 : 1;  // f16 halves of q and of the probabilities
  // How far a tile's largest value scale may be above the smallest so far before its probabilities are lifted.
  static constexpr float kRaised = sizeof(T) == 4 ? 2.0f : 32.0f;
  static constexpr int kFragments = S::kSteps * NT * kHalves;  // of q
  static constexpr int kQBytes = Q_SMEM ? kFragments * 256 : 0;
  unsigned q[Q_SMEM ? 1 : kFragments][2];
  unsigned q_at;  // Q_SMEM: where this lane's are
  static constexpr int fragment_of(int ks, int nt, int h) { return (ks * NT + nt) * kHalves + h; }
  __device__ __forceinline__ void put_q(int i, unsigned b0, unsigned b1) {
    if constexpr (Q_SMEM) {
      asm volatile("st.shared.v2.u32 [%0], {%1,%2};\n" ::"r"(q_at + i * 256), "r"(b0), "r"(b1) : "memory");
    } else {
      q[i][0] = b0;
      q[i][1] = b1;
    }
  }
  __device__ __forceinline__ Words<2> get_q(int i) const {
    Words<2> b;
    if constexpr (Q_SMEM) {
      load_words(b, q_at + i * 256);
    } else {
      b.w[0] = q[i][0];
      b.w[1] = q[i][1];
    }
    return b;
  }
  float by[NT][2];  // what takes the column's sums of codes to scores in the log2 domain
  // Whether sums of codes, below 2^31, times `by` may pass f32's range: a small key scale goes first then.
  __device__ __forceinline__ bool wide() const {
    float t = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) t = fmaxf(t, fmaxf(fabsf(by[nt][0]), fabsf(by[nt][1])));
    return t > 0x1p90f;
  }
  unsigned k_at, v_at[2];  // this lane's offsets: of row g = lane / 4 of K; of rows g = 2 (lane % 4), and one more, of V

  __device__ __forceinline__ explicit Warp8(int lane) {
    k_at = place<D, KT>(key_of<D>(lane / 4), lane & 3);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = key_of<D>((lane & 3) * 2 + i);
      v_at[i] = S::kBytes == 16 ? place<D, KT>(r, lane / 4) : place<D, KT>(r, lane / 8) + (lane / 4 & 1) * 8;
    }
  }

  // rows: q's rows of the block in shared memory, ROW bytes apart; this warp's begin at row0
  template <int ROW>
  __device__ __forceinline__ void load_q(unsigned rows, int lane, int row0, float scale_log2) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const unsigned p = rows + (row0 + nt * 8 + lane / 4) * ROW;
      // step ks of 64-element group ks / 4: elements (lane % 4) * 16 + ks % 4 * 4 .. + 4 of the group
      float x[S::kSteps][4], top = 0.0f;
#pragma unroll
      for (int ks = 0; ks < S::kSteps; ++ks) {
        Words<sizeof(T)> e;  // four elements
        load_words(e, p + ((ks >> 2) * 64 + (lane & 3) * 16 + (ks & 3) * 4) * static_cast<int>(sizeof(T)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 2) x[ks][i] = __uint_as_float(i & 1 ? e.w[i / 2] & 0xffff0000u : e.w[i / 2] << 16);
          else x[ks][i] = __uint_as_float(e.w[i]);
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
      for (int ks = 0; ks < S::kSteps; ++ks) {
        unsigned hi[2], lo[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const float u = x[ks][2 * b] * f, v = x[ks][2 * b + 1] * f;
          hi[b] = f16x2(u, v);
          const float2 h = f32x2(hi[b]);
          lo[b] = f16x2(u - h.x, v - h.y);
        }
        put_q(fragment_of(ks, nt, 0), hi[0], hi[1]);
        if constexpr (kHalves == 2) put_q(fragment_of(ks, nt, 1), lo[0], lo[1]);
      }
    }
    __syncwarp();
  }

  // s = K Q^T of the tile, as sums of codes
  __device__ __forceinline__ void scores(float (&s)[KT][NT][4], unsigned k_tile) const {
    // the tensor cores cut the low bits of a running sum: f32's are taken over 64 elements; bf16's in two chains, for the
    // products' latency
    float t[KT][NT][4];
#pragma unroll
    for (int g = 0; g < D / 64; ++g) {
      unsigned a[KT][4][4];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        Words<4> lo, hi;
        const unsigned at = k_tile + kt * kSub * S::kRow + (k_at ^ ((g & 1) << 6)) + (g >> 1) * S::kPart;
        load_words(lo, at);
        load_words(hi, at + 8 * S::kRow);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[kt][i][0] = codes_f16x2(lo.w[i], 0);
          a[kt][i][1] = codes_f16x2(hi.w[i], 0);
          a[kt][i][2] = codes_f16x2(lo.w[i], 2);
          a[kt][i][3] = codes_f16x2(hi.w[i], 2);
        }
      }
#pragma unroll
      for (int h = kHalves - 1; h >= 0; --h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const Words<2> b = get_q(fragment_of(g * 4 + i, nt, h));
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              float (&to)[4] = kHalves == 2 ? (g > 0 ? t[kt][nt] : s[kt][nt]) : g & 1 ? t[kt][nt] : s[kt][nt];
              const bool first = i == 0 && h == kHalves - 1 && (kHalves == 2 || g < 2);
              if (first) mma_f16_first(to, a[kt][i], b.w[0], b.w[1]);
              else mma_f16(to, a[kt][i], b.w[0], b.w[1]);
            }
          }
      if (kHalves == 2 ? g > 0 : D > 64 && g == D / 64 - 1) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) s[kt][nt][j] += t[kt][nt][j];
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

  // Brings a score tile's probabilities near the top of f16's range, by a power of two of the column.  `of` becomes what
  // takes the sums of products back, times `by`.
  static __device__ __forceinline__ void lift(float (&s)[NT][4], float by, float (&of)[NT][2]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float t = fmaxf(s[nt][j], s[nt][j + 2]);
        t = fmaxf(t, __shfl_xor_sync(kFull, t, 4));
        t = fmaxf(t, __shfl_xor_sync(kFull, t, 8));
        t = fmaxf(t, __shfl_xor_sync(kFull, t, 16));
        // to [2^14, 2^15)
        const int up = t > 0.0f ? min(max(14 + 127 - (__float_as_int(t) >> 23), 0), 120) : 0;
        const float f = __int_as_float((127 + up) << 23);
        of[nt][j] = by * __int_as_float((127 - up) << 23);
        s[nt][j] *= f;
        s[nt][j + 2] *= f;
      }
  }

  // This lane's part of 16 values: kBytes neighbouring elements of four keys.
  struct V {
    Words<S::kBytes / 4> r[4];
    __device__ __forceinline__ void load(const Warp8 &w, unsigned v_tile, int piece) {
#pragma unroll
      for (int i = 0; i < 4; ++i) load_words(r[i], v_tile + w.v_at[i & 1] + (i >> 1) * 8 * S::kRow + piece * S::kPart);
    }
    // keys outside [k0, k1) as zeros
    __device__ __forceinline__ void keep(int k0, int k1, int lane) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int key = key_of<D>((lane & 3) * 2 + (i & 1)) + (i >> 1) * 8;
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
  // y = V^T P^T (first) or y += V^T P^T
  static __device__ __forceinline__ void weigh(float (&y)[4], const unsigned (&a)[4], const P &p, int nt, bool first) {
#pragma unroll
    for (int h = kHalves - 1; h >= 0; --h)
      if (first && h == kHalves - 1) mma_f16_first(y, a, p.b[nt][h][0], p.b[nt][h][1]);
      else mma_f16(y, a, p.b[nt][h][0], p.b[nt][h][1]);
  }
};

// A variant: NT 8-row tiles of a warp, RW warps that share their tiles, each with rows of its own, WARPS of a CTA beside
// the FEED that feed them, KT matrix tiles of 16 keys in a step, CTAS on an SM.  BOXED: pages hold whole groups of 8 keys.
template <typename T_, int D_, int NT_, int RW_, int WARPS_, int FEED_, int KT_, int CTAS_, bool BOXED_, bool Q_SMEM_ = false>
struct Pick8 {
  using T = T_;
  using S = Shape8<D_, KT_>;
  static constexpr int D = D_, NT = NT_, RW = RW_, WARPS = WARPS_, FEED = FEED_, KT = KT_, CTAS = CTAS_;
  static constexpr bool BOXED = BOXED_;
  using W = Warp8<T_, D_, NT_, KT_, Q_SMEM_>;
  static constexpr int rows = NT * RW * 8, ctas = kSms * CTAS, threads = 32 * (WARPS + FEED);
  // items that are known ahead, with their q
  static constexpr int q_row = D * static_cast<int>(sizeof(T)) + 16, q_bytes = rows * q_row, slots = q_bytes <= 2400 ? 4 : q_bytes <= 4800 ? 3 : 2;
  // beside a stage: the scales of its groups of 8 keys (of its keys), and of their values
  static constexpr int groups = BOXED ? KT * 2 : S::kTile, scales = 2 * groups * 4;
  // a row group's sums at a job's end, as its warps have them in registers: those of values, of probabilities, and the maximum
  static constexpr int join_bytes = RW * (D / 16 * 4 + 4) * NT * 128;
  static constexpr int fragment_bytes = slots * RW * W::kQBytes;
  static constexpr int fixed = join_bytes + slots * q_bytes + fragment_bytes;
  // the ring has what the SM's shared memory holds beside that and the static part
  static constexpr int fit = (228 * 1024 / CTAS - 1024 - 1024 - 512 - 64 * WARPS * NT - 24 * 32 - fixed) / (S::kStage + scales);
  // A stage is always filled by the same warp and emptied by the same group: waits tell two phases of a barrier apart, and
  // who let one pass would take the next but one for it.
  static constexpr int turn = std::lcm(WARPS / RW, FEED), STAGES = (fit < 32 ? fit : 32) / turn * turn;
  static constexpr int smem = 1024 + STAGES * (S::kStage + scales) + fixed;  // stages begin at multiples of 1024
  static_assert(STAGES > WARPS / RW && STAGES % (WARPS / RW) == 0 && STAGES % FEED == 0, "two stages per key group at least");
  static_assert(FEED <= 8 && (FEED & (FEED - 1)) == 0, "a batch of the feeding warps' boxes holds a multiple of FEED tiles");
};

// An item, or the part of it that lies in a CTA's share, as the feeding warps tell the others.
struct Job {
  int k0, k1;           // its keys
  int t0, tokens, len;  // its request's rows of q, and keys
  int rows, head, block;
  int slot;   // where its sums go in the workspace; -1: it lies in this CTA, and its results go to the output
  int last;   // the last CTA that has a part of it, where it begins in this one; else -1
  int none;   // there is none any more
};

// What the feeding warps and the others share beside the ring: shared-memory addresses.
struct Ring {
  unsigned stages, scales, q, fragments, missing;
  unsigned full, empty, job_full, job_empty, turn;  // of barriers: of a stage, of a job's slot, of a key group's turn to join
  Job *jobs;
  volatile int *failed;  // a wait of a warp ran out
};

// A warp whose wait ran out tells the others, which then stop at the next wait that they would have to wait at.
__device__ __forceinline__ void give_up(const Ring &ring) {
  if ((threadIdx.x & 31) == 0) {
    *ring.failed = 1;
    report(GDN_DEVICE_WAIT_TIMEOUT);
  }
  __syncwarp();
}

// A feeding warp: puts every FEED-th tile of the share's items into the ring, and the last one the items themselves.
// (One alone takes 600 to 1000 clocks for a tile, all latency: waits, exchanges of lanes, 60 to 80 to issue a tensor copy.)
template <typename P>
struct Feed {
  using T = typename P::T;
  using S = typename P::S;
  static constexpr int D = P::D, kTile = S::kTile;
  using Part = Item<P::rows, 1, kTile>;
  const Call &c;
  const Ring &ring;
  int lane, id;
  int stage, slot = 0;
  int skip;  // tiles before this warp's next one, from the item's first
  unsigned phase = 1, job_phase = 1;
  bool filled = false, slots_filled = false;  // every stage, every slot has been

  __device__ __forceinline__ Feed(const Call &c_, const Ring &r) : c(c_), ring(r), lane(threadIdx.x & 31), id((threadIdx.x >> 5) - P::WARPS), stage(id), skip(id) {}

  __device__ __forceinline__ bool wait(unsigned bar, unsigned of) {
    if (mbar_wait<(P::NT > 1)>(bar, of, c.wait_clocks, ring.failed)) return true;
    give_up(ring);
    drain();
    return false;
  }
  // This warp's copies have to land before the CTA ends, whatever has become of the warps that take them.
  __device__ __forceinline__ void drain() {
#pragma unroll 1
    for (int x = id; x < P::STAGES; x += P::FEED)
      if (x < stage || filled) mbar_wait<(P::NT > 1)>(ring.full + x * 8, x < stage ? phase ^ 1 : phase, kWaitClocks, nullptr);
    asm volatile("cp.async.wait_all;\n" ::: "memory");
    if (id == P::FEED - 1)
#pragma unroll 1
      for (int x = 0; x < P::slots; ++x)
        if (x < slot || slots_filled) mbar_wait<(P::NT > 1)>(ring.job_full + x * 8, x < slot ? job_phase ^ 1 : job_phase, kWaitClocks, nullptr);
  }
  // The item at unit u as a job, and its rows of q: row n is token n / group, query head n % group of the key head; zeros
  // for those that are not.
  __device__ __forceinline__ bool put_job(const Share &sh, const Part &f, int head, long long u) {
    if (id != P::FEED - 1) return true;  // (the other one has the first tile meanwhile)
    if (!wait(ring.job_empty + slot * 8, job_phase)) return false;
    const int block = f.item - head * f.r.blocks, rows = f.r.tokens * static_cast<int>(c.group);
    if (lane == 0) {
      Job &j = ring.jobs[slot];
      j.k0 = f.k0;
      j.k1 = f.k1;
      j.t0 = f.r.t0;
      j.tokens = f.r.tokens;
      j.len = f.r.len;
      j.rows = rows;
      j.head = head;
      j.block = block;
      j.none = 0;
      const bool whole = f.tile0 == 0 && f.tile1 == f.r.tiles;
      j.slot = whole ? -1 : 2 * sh.cta + (u == sh.u0 ? 0 : 1);  // an item that goes on from the CTA before is the share's first
      j.last = -1;
      if (!whole && f.tile0 == 0) {
        const long long end = u + f.units + (f.r.tiles - f.tile1) - 1;  // the item's last unit
        j.last = static_cast<int>(((end + 1) * sh.ctas - 1) / sh.total);
      }
      mbar_arrive(ring.job_full + slot * 8);
    }
    if (f.k0 < f.k1) {
      const unsigned to = ring.q + slot * P::q_bytes;
      auto copy = [&](auto bytes) {
        constexpr int kBytes = bytes(), kOf = D * static_cast<int>(sizeof(T)) / kBytes;
#pragma unroll 4
        for (int x = lane; x < P::rows * kOf; x += 32) {
          const int n = x / kOf, col = x % kOf * kBytes, row = block * P::rows + n, t = c.group_div.div(row);
          const char *src = static_cast<const char *>(c.q);
          if (row < rows)
            src += (static_cast<int64_t>(f.r.t0 + t) * c.q_stride + (static_cast<int64_t>(head) * c.group + (row - t * static_cast<int>(c.group))) * D) *
                       static_cast<int>(sizeof(T)) + col;
          const int size = row < rows ? kBytes : 0;
          const unsigned dst = to + n * P::q_row + col;
          if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(dst), "l"(src), "r"(size) : "memory");
          else asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(size) : "memory");
        }
      };
      if (c.q_wide) copy(std::integral_constant<int, 16>{});
      else copy(std::integral_constant<int, 4>{});
    }
    next_job();
    return true;
  }
  // After the last item.
  __device__ __forceinline__ void put_end() {
    if (id == P::FEED - 1) {
      if (!wait(ring.job_empty + slot * 8, job_phase)) return;
      if (lane == 0) {
        ring.jobs[slot].none = 1;
        mbar_arrive(ring.job_full + slot * 8);
      }
      next_job();
    }
    drain();
  }
  __device__ __forceinline__ void next_job() {
    mbar_arrive_after_copies(ring.job_full + slot * 8);
    if (++slot == P::slots) {
      slot = 0;
      job_phase ^= 1;
      slots_filled = true;
    }
  }
  __device__ __forceinline__ void next_stage() {
    stage += P::FEED;
    if (stage >= P::STAGES) {
      stage -= P::STAGES;
      phase ^= 1;
      filled = true;
    }
  }
  // Past an item of n tiles.
  __device__ __forceinline__ void next_item(int n) { skip = (skip + P::FEED - n % P::FEED) % P::FEED; }
};

// Boxes of c.box rows of a page by tensor copies.  A lane has one box of 32: its page, the place in it and its scales,
// the pages looked up two such batches ahead and the scales one.
template <typename P>
__device__ __forceinline__ void feed_boxes(const Call &c, const CUtensorMap *k_map, const CUtensorMap *v_map, const Share &sh, uint32_t seq,
                                           long long in_seq, const Request &first, const Ring &ring) {
  using S = typename P::S;
  constexpr int kTile = S::kTile, kMost = kTile / 8;  // boxes of a tile
  Feed<P> d(c, ring);
  const int lane = d.lane, box = c.box, per_tile = kTile / box, batch = 32 * box;
  typename Feed<P>::Part f;
  f.seq = seq;
  f.in_seq = in_seq;
  f.r = first;
  long long u = sh.u0;
  // of a batch: this lane's box's page, or -1 where there is none, and its scales; what an item begins with is found while the
  // one before is fed
  auto page_of = [&](const typename Feed<P>::Part &x, int key) {
    return key < x.k1 ? c.table[static_cast<uint64_t>(x.seq) * c.max_pages + c.page_div.div(key)] : -1;
  };
  auto scale_of = [&](const float *scales, int page, int head) {
    return static_cast<uint32_t>(page) < c.n_pages ? scales[static_cast<uint64_t>(page) * c.n_kv + head] : 0.0f;
  };
  bool more = f.find(c, u, sh.u1);
  if (!more) {
    d.put_end();
    return;
  }
  int page = page_of(f, f.k0 + lane * box), page1 = page_of(f, f.k0 + batch + lane * box);
  float ks = 0.0f, vs = 0.0f;
  while (more) {
    typename Feed<P>::Part g = f;
    int g_page = -1, g_page1 = -1;
    const int head = f.item / f.r.blocks;
    if (!d.put_job(sh, f, head, u)) return;
    ks = scale_of(c.k_scale, page, head);
    vs = scale_of(c.v_scale, page, head);
    bool looked = false;
    auto look_ahead = [&] {
      looked = true;
      g.pass(u);
      more = g.find(c, u, sh.u1);
      if (more) {
        g_page = page_of(g, g.k0 + lane * box);
        g_page1 = page_of(g, g.k0 + batch + lane * box);
      }
    };
    for (int b0 = f.k0; b0 < f.k1; b0 += batch) {
      const int key = b0 + lane * box;
      const int at = key - static_cast<int>(c.page_div.div(key) * c.page_size);
      const bool there = static_cast<uint32_t>(page) < c.n_pages;
      const unsigned valid = __ballot_sync(kFull, there);
      const unsigned gone = __ballot_sync(kFull, !there && key < f.k1 && key + box > f.r.first);
      const int page2 = page_of(f, key + 2 * batch);
      const float ks1 = scale_of(c.k_scale, page1, head), vs1 = scale_of(c.v_scale, page1, head);
#pragma unroll 1
      for (int x = d.skip * per_tile; x < 32 && b0 + x * box < f.k1; x += P::FEED * per_tile) {
        const unsigned of_tile = ((2u << (per_tile - 1)) - 1) << x;
        const unsigned full = ring.full + d.stage * 8, to = ring.stages + d.stage * S::kStage;
        int pg[kMost], row[kMost];
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
          pg[i] = __shfl_sync(kFull, page, x + i);
          row[i] = __shfl_sync(kFull, at, x + i);
        }
        if (!d.wait(ring.empty + d.stage * 8, d.phase)) return;
        if (lane == 0) mbar_expect(full, __popc(valid & of_tile) * box * 2 * P::D);
        // boxes past the item's end, or of no page, are left as they are and cut out later
        if (elected()) {
#pragma unroll
          for (int i = 0; i < kMost; ++i)
            if (valid & of_tile & 1u << (x + i & 31)) {
              const unsigned dst = to + i * box * S::kRow;
#pragma unroll
              for (int e = 0; e < S::kParts; ++e) {
                copy_box(dst + e * S::kPart, k_map, e * 128, row[i], head, pg[i], full);
                copy_box(dst + S::kCodes + e * S::kPart, v_map, e * 128, row[i], head, pg[i], full);
              }
            }
        }
        {  // lane i has the scales of the tile's group i of 8 keys
          const int i = x + (lane & (P::groups - 1)) * 8 / box;
          const float of_k = __shfl_sync(kFull, ks, i), of_v = __shfl_sync(kFull, vs, i);
          if (lane < P::groups) {
            const unsigned dst = ring.scales + d.stage * P::scales + lane * 4;
            asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(dst), "f"(of_k) : "memory");
            asm volatile("st.shared.f32 [%0], %1;\n" ::"r"(dst + P::groups * 4), "f"(of_v) : "memory");
          }
          if (lane == 0) asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(ring.missing + d.stage * 4), "r"(gone & of_tile) : "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(full);
        }
        d.next_stage();
        if (!looked) look_ahead();
      }
      page = page1;
      page1 = page2;
      ks = ks1;
      vs = vs1;
    }
    if (!looked) look_ahead();
    d.next_item((f.k1 - f.k0 + kTile - 1) / kTile);
    f = g;
    page = g_page;
    page1 = g_page1;
  }
  d.put_end();
}

// Row by row, for pages of any size: a lane has a key of the tile.
template <typename P>
__device__ __forceinline__ void feed_rows(const Call &c, const Share &sh, uint32_t seq, long long in_seq, const Request &first, const Ring &ring) {
  using S = typename P::S;
  constexpr int D = P::D, kTile = S::kTile;
  constexpr int kChunks = D / 16;                  // 16-byte chunks per row
  constexpr int kPer = 32 / kChunks;               // rows one access of the warp covers
  constexpr int kAccesses = kTile * kChunks / 32;  // of K or V
  Feed<P> d(c, ring);
  const int lane = d.lane, my_row = lane / kChunks, my_chunk = lane % kChunks;
  const unsigned mine = place<D, P::KT>(my_row, my_chunk);
  const char *const k = static_cast<const char *>(c.k) + my_chunk * 16, *const v = static_cast<const char *>(c.v) + my_chunk * 16;
  typename Feed<P>::Part f;
  f.seq = seq;
  f.in_seq = in_seq;
  f.r = first;
  for (long long u = sh.u0; f.find(c, u, sh.u1); f.pass(u)) {
    const int head = f.item / f.r.blocks;
    const int32_t *const table = c.table + static_cast<uint64_t>(f.seq) * c.max_pages;
    if (!d.put_job(sh, f, head, u)) return;
    int key = f.k0 + d.skip * kTile + (lane & (kTile - 1));
    int page = key < f.k1 ? table[c.page_div.div(key)] : 0;
    for (int tile = f.k0 + d.skip * kTile; tile < f.k1; tile += P::FEED * kTile) {
      const int ahead = key + P::FEED * kTile, next = ahead < f.k1 ? table[c.page_div.div(ahead)] : 0;
      const bool none = static_cast<uint32_t>(page) >= c.n_pages, valid = key < f.k1 && !none;
      const bool gone = __any_sync(kFull, none && key < f.k1 && key >= f.r.first);
      const int o = key - static_cast<int>(c.page_div.div(key) * c.page_size);
      const long long row_at = valid ? page * c.page_stride + head * c.head_stride + o * c.slot_stride : -1;  // -1: zeros
      const uint64_t scale_at = (valid ? static_cast<uint64_t>(page) * c.n_kv : 0) + head;
      const unsigned full = ring.full + d.stage * 8, to = ring.stages + d.stage * S::kStage;
      if (!d.wait(ring.empty + d.stage * 8, d.phase)) return;
      if (lane < kTile) {
        const unsigned dst = ring.scales + d.stage * P::scales + lane * 4;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst), "l"(c.k_scale + scale_at) : "memory");
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;\n" ::"r"(dst + kTile * 4), "l"(c.v_scale + scale_at) : "memory");
      }
      if (lane == 0) {
        asm volatile("st.shared.u32 [%0], %1;\n" ::"r"(ring.missing + d.stage * 4), "r"(static_cast<unsigned>(gone)) : "memory");
        mbar_arrive(full);
      }
#pragma unroll
      for (int x = 0; x < kAccesses; ++x) {
        const int row = x * kPer;  // behind my_row
        const long long off = __shfl_sync(kFull, row_at, my_row + row);
        const long long from = off < 0 ? 0 : off;
        const unsigned dst = to + (mine ^ (order<D>(row) << 4)) + row * S::kRow;
        cp_async_16_or_zero(dst, k + from, off >= 0);
        cp_async_16_or_zero(dst + S::kCodes, v + from, off >= 0);
      }
      mbar_arrive_after_copies(full);
      d.next_stage();
      key = ahead;
      page = next;
    }
    d.next_item((f.k1 - f.k0 + kTile - 1) / kTile);
  }
  d.put_end();
}

template <typename P>
__global__ void __launch_bounds__(P::threads, P::CTAS) gdn_attn_fp8_kernel(const __grid_constant__ Call c, const __grid_constant__ CUtensorMap k_map,
                                                                             const __grid_constant__ CUtensorMap v_map) {
  using T = typename P::T;
  constexpr int D = P::D, NT = P::NT, RW = P::RW, WARPS = P::WARPS, KT = P::KT;
  using S = Shape8<D, KT>;
  using W = typename P::W;
  constexpr int kTile = S::kTile;
  constexpr int kRows = P::rows;       // rows of a block
  constexpr int KW = WARPS / RW;       // key groups: group g takes every KW-th tile of the share
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ long long s_scan[WARPS + P::FEED], s_offset;
  __shared__ uint32_t s_seq;
  __shared__ Request s_first;
  __shared__ unsigned s_bad[RW];
  __shared__ unsigned s_missing[P::STAGES];
  __shared__ alignas(8) uint64_t s_full[P::STAGES], s_empty[P::STAGES], s_job_full[P::slots], s_job_empty[P::slots], s_turn[WARPS];
  __shared__ Job s_jobs[P::slots];
  __shared__ int s_failed;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned start = (1024u - (smem_u32(smem) & 1023u)) & 1023u;
  float4 *join = reinterpret_cast<float4 *>(smem + start + P::STAGES * (S::kStage + P::scales));
  const Ring ring{smem_u32(smem) + start, smem_u32(smem) + start + P::STAGES * S::kStage, smem_u32(join) + P::join_bytes, smem_u32(join) + P::join_bytes + P::slots * P::q_bytes,
                  smem_u32(s_missing), smem_u32(s_full), smem_u32(s_empty), smem_u32(s_job_full), smem_u32(s_job_empty), smem_u32(s_turn), s_jobs, &s_failed};
  if (tid < P::STAGES) {
    mbar_init(ring.full + tid * 8, P::BOXED ? 2 : 33);  // what the feeding warp stores, and its copies
    mbar_init(ring.empty + tid * 8, RW);
  }
  if (tid < P::slots) {
    mbar_init(ring.job_full + tid * 8, 33);
    mbar_init(ring.job_empty + tid * 8, WARPS);
  }
  if (tid < WARPS) mbar_init(ring.turn + tid * 8, 1);
  if (tid == 0) s_failed = 0;
  asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");

  begin_in_order();
  // what the join finds in the place of a part that is not put because a wait ran out: rows of NaN
  if (!c.whole_items)
    for (int i = tid; i < 2 * kRows; i += P::threads) c.part_ml[static_cast<size_t>(2) * blockIdx.x * kRows + i] = make_float2(0.0f, NAN);
  const Share sh = take_share<kRows, WARPS + P::FEED>(c, s_scan, s_seq, s_offset, &s_first);  // (its barriers show the initialised ones)
  if (sh.cta >= sh.ctas) return;
  if (warp >= WARPS) {
    if constexpr (P::BOXED) feed_boxes<P>(c, &k_map, &v_map, sh, s_seq, s_offset, s_first, ring);
    else feed_rows<P>(c, sh, s_seq, s_offset, s_first, ring);
    return;
  }
  const int kg = warp / RW, rg = warp % RW, row0 = rg * NT * 8;  // key group; rows of the block
  W w(lane);
  int slot = 0, stage = kg;
  int ahead = kg;  // tiles until this group's next one, from the job's first
  unsigned phase = 0, job_phase = 0, turn_phase = 0;
  // Where a wait runs out the warp ends, and with it, at the next turns that it does not give, all that its row group would put.
  auto wait = [&](unsigned bar, unsigned of) {
    const bool ended = mbar_wait<(P::NT > 1)>(bar, of, c.wait_clocks, ring.failed);
    if (!ended) give_up(ring);
    return ended;
  };
  while (true) {
    if (!wait(ring.job_full + slot * 8, job_phase)) return;
    const Job &job = s_jobs[slot];
    if (job.none) break;
    // the last key each of this lane's columns sees, and keys that every row of this warp does: [all0, all1)
    int last[NT][2];
    const int first_row = job.block * kRows + row0, before = job.len - job.tokens, k1 = job.k1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) last[nt][j] = before + static_cast<int>(c.group_div.div(min(first_row + nt * 8 + (lane & 3) * 2 + j, job.rows - 1)));
    const int last0 = before + static_cast<int>(c.group_div.div(min(first_row, job.rows - 1)));  // of the first and the last row
    const int last1 = before + static_cast<int>(c.group_div.div(min(first_row + NT * 8, job.rows) - 1));
    const int all1 = min(last0 + 1, k1), all0 = c.window ? less_window(last1 + 1, c.window) : 0;

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

    const int n_tiles = (k1 - job.k0 + kTile - 1) / kTile;
    int key0 = job.k0 + ahead * kTile;
    bool bad_page = false;
    unsigned least_scale = 0x7f800000u;  // of the job's values so far (of this key group): an f32's bits
    // (every key group puts the same fragments)
    w.q_at = ring.fragments + (slot * RW + rg) * W::kQBytes + lane * 8;
    if (ahead < n_tiles) w.template load_q<P::q_row>(ring.q + slot * P::q_bytes, lane, row0, c.scale_log2);
#pragma unroll 1
    for (; ahead < n_tiles; ahead += KW, key0 += kTile * KW) {
      if (!wait(ring.full + stage * 8, phase)) return;
      const unsigned k_tile = ring.stages + stage * S::kStage, v_tile = k_tile + S::kCodes, scales = ring.scales + stage * P::scales;
      bad_page |= s_missing[stage] != 0u;
      // the tile is done with: the next of this group
      auto leave = [&] {
        __syncwarp();
        if (lane == 0) mbar_arrive(ring.empty + stage * 8);
        stage += KW;
        if (stage >= P::STAGES) {
          stage -= P::STAGES;
          phase ^= 1;
        }
      };
      // scores
      float s[KT][NT][4];
      const bool edge = key0 + kTile > all1 || key0 < all0;
      // keys that a row of this warp sees, of the tile
      const int seen0 = edge && c.window ? max(0, less_window(last0 + 1 - key0, c.window)) : 0;
      const int seen1 = edge ? min(min(last1 + 1, k1) - key0, kTile) : kTile;
      w.scores(s, k_tile);
      float vs[KT][2];  // the scales of the values of this lane's keys; BOXED: of these groups of 8 keys
      unsigned most = 0u, least = 0xffffffffu;  // of those that a row sees
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int from = kt * kSub + h * 8, key = from + (P::BOXED ? 0 : key_of<D>(lane / 4)), at = P::BOXED ? kt * 2 + h : key;
          float ks = load_f32(scales + at * 4);
          if (w.wide() && fabsf(ks) < 1.0f) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) s[kt][nt][2 * h + j] *= ks;
            ks = 1.0f;
          }
          vs[kt][h] = load_f32(scales + (P::groups + at) * 4);
          if (!edge || (key + (P::BOXED ? 7 : 0) >= seen0 && key < seen1)) {
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
              const int key = key0 + kt * kSub + key_of<D>(lane / 4) + (j >> 1) * 8, hi = min(last[nt][j & 1], k1 - 1);
              const long long lo = c.window ? static_cast<long long>(last[nt][j & 1]) - c.window : -1;
              if (key > hi || key <= lo) s[kt][nt][j] = -INFINITY;
            }
      }
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
      if constexpr (!P::BOXED) {
        most = __reduce_max_sync(kFull, most);
        least = __reduce_min_sync(kFull, least);
      }
      const float ref = __uint_as_float(most);
      bool apart = !(most < 0x7f800000u && __uint_as_float(least) * 256.0f >= ref) && most != 0u;
      if (most != least && !apart) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float by = most ? vs[kt][h] / ref : 0.0f;  // a key that no row sees has the probability 0
            const bool use = most && by >= 0.0f && by <= 1.0f;  // (what no row sees may have any scale)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 2; ++j) s[kt][nt][2 * h + j] = use ? s[kt][nt][2 * h + j] * by : 0.0f;
          }
      }
      // Whether what f16 cuts off small probabilities may show in this tile's values.
      least_scale = most > 0x7f800000u ? 0u : min(least_scale, least);  // (0: none that could be compared with)
      const bool raised = ref > __uint_as_float(least_scale) * W::kRaised;
      // output
      if (!edge && !apart && !raised) {
        typename W::P p[KT];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) p[kt].take(s[kt]);
#pragma unroll
        for (int x = 0; x < S::kParts; ++x) {
          typename W::V v[KT];
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) v[kt].load(w, v_tile + kt * kSub * S::kRow, x);
#pragma unroll
          for (int md = 0; md < S::kBytes / 2; ++md) {
            float y[NT][4];
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
              unsigned a[4];
              v[kt].fragment(a, md);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) W::weigh(y[nt], a, p[kt], nt, kt == 0);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[x * (S::kBytes / 2) + md][nt][j] += ref * y[nt][j];
          }
        }
        leave();
        continue;
      }
      // A key that a token does not see must not reach its row even as 0 * v (v may be stale or NaN).  Keys that no
      // token of the warp sees are cut out of V; if tokens see different keys of the tile and one of those is NaN, or the
      // scales are apart, each token's columns take products of their own, in the latter case 8 keys (or a page's) a time.
      // Where the scales are apart or raised, the probabilities of such a product are lifted.
      const bool folded = !apart;
      if (folded && last0 != last1) {
        bool nan = false;
#pragma unroll 1
        for (int x = 0; x < S::kParts * KT; ++x) {
          typename W::V v;
          v.load(w, v_tile + x % KT * kSub * S::kRow, x / KT);
          v.keep(seen0 - x % KT * kSub, seen1 - x % KT * kSub, lane);
          nan |= v.has_nan();
        }
        apart = __any_sync(kFull, nan);
      }
#pragma unroll 1
      for (int sees = apart ? last0 : last1; sees <= last1; ++sees) {  // the last key that the token sees
        const int end = apart ? min(min(sees + 1, k1) - key0, kTile) : seen1;
        int from = !apart ? seen0 : c.window ? max(0, less_window(sees + 1 - key0, c.window)) : 0;
#pragma unroll 1
        while (from < end) {
          int to = min(end, (from / kSub + 1) * kSub);
          const int kt0 = from / kSub;
          if (!folded) {
            if constexpr (P::BOXED) {
              to = min(to, (from / 8 + 1) * 8);
            } else {
              const int key = key0 + from;
              to = min(to, from + static_cast<int>(c.page_size) - (key - static_cast<int>(c.page_div.div(key) * c.page_size)));
            }
          }
          float ps[NT][4], of[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            of[nt][0] = of[nt][1] = ref;
#pragma unroll
            for (int j = 0; j < 4; ++j) ps[nt][j] = KT > 1 && kt0 > 0 ? s[KT - 1][nt][j] : s[0][nt][j];
          }
          if (!folded || raised) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int key = kt0 * kSub + key_of<D>(lane / 4) + (j >> 1) * 8;
                if (key < from || key >= to) ps[nt][j] = 0.0f;
              }
            W::lift(ps, folded ? ref : load_f32(scales + (P::groups + (P::BOXED ? from / 8 : from)) * 4), of);
          }
          typename W::P pk;
          pk.take(ps);
#pragma unroll
          for (int x = 0; x < S::kParts; ++x) {
            typename W::V v;
            v.load(w, v_tile + kt0 * kSub * S::kRow, x);
            v.keep(from - kt0 * kSub, to - kt0 * kSub, lane);
#pragma unroll
            for (int md = 0; md < S::kBytes / 2; ++md) {
              unsigned a[4];
              v.fragment(a, md);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float y[4];
                W::weigh(y, a, pk, nt, true);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  if (!apart || last[nt][j & 1] == sees) acc[x * (S::kBytes / 2) + md][nt][j] += of[nt][j & 1] * y[j];
              }
            }
          }
          from = to;
        }
      }
      leave();
    }
    ahead -= n_tiles;

    // Join the key groups, one after the other, each adding its sums to those before, first the one whose last tile came
    // first (so the order goes by the sizes alone); the last one puts the results.
    const int turn = ahead;
    const unsigned turns = ring.turn + rg * KW * 8;
    if (!wait(turns + (KW - 1) * 8, turn_phase ^ 1)) return;  // the join of the job before is over (else a turn of that one would pass for this one's)
    if (turn && !wait(turns + (turn - 1) * 8, turn_phase)) return;
    turn_phase ^= 1;
    bad_page = __any_sync(kFull, bad_page) || (turn && s_bad[rg]);
    float4 *const sums = join + rg * (P::join_bytes / RW / 16) + lane;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float4 *const of = sums + nt * (D / 16 + 1) * 32;
      if (turn) {
        const float4 b = of[D / 16 * 32];
        const float t0 = fmaxf(m[nt][0], b.x), t1 = fmaxf(m[nt][1], b.y);
        const float g0 = exp2_fast(m[nt][0] - t0), g1 = exp2_fast(m[nt][1] - t1), h0 = exp2_fast(b.x - t0), h1 = exp2_fast(b.y - t1);
        m[nt][0] = t0;
        m[nt][1] = t1;
        l[nt][0] = l[nt][0] * g0 + b.z * h0;
        l[nt][1] = l[nt][1] * g1 + b.w * h1;
#pragma unroll
        for (int md = 0; md < D / 16; ++md) {
          const float4 y = of[md * 32];
          acc[md][nt][0] = acc[md][nt][0] * g0 + y.x * h0;
          acc[md][nt][1] = acc[md][nt][1] * g1 + y.y * h1;
          acc[md][nt][2] = acc[md][nt][2] * g0 + y.z * h0;
          acc[md][nt][3] = acc[md][nt][3] * g1 + y.w * h1;
        }
      }
      if (turn < KW - 1) {
        of[D / 16 * 32] = make_float4(m[nt][0], m[nt][1], l[nt][0], l[nt][1]);
#pragma unroll
        for (int md = 0; md < D / 16; ++md) of[md * 32] = make_float4(acc[md][nt][0], acc[md][nt][1], acc[md][nt][2], acc[md][nt][3]);
      }
    }
    if (lane == 0 && turn < KW - 1) s_bad[rg] = bad_page;
    __syncwarp();
    if (lane == 0) mbar_arrive(turns + turn * 8);
    if (turn == KW - 1) {
      if (bad_page && lane == 0) report(GDN_DEVICE_BAD_PAGE);
      // column 2 (lane % 4) + j of the tile is a row; this lane has kBytes neighbouring elements of every 128 (64) of it
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float den = l[nt][j];
          den += __shfl_xor_sync(kFull, den, 4);
          den += __shfl_xor_sync(kFull, den, 8);
          den += __shfl_xor_sync(kFull, den, 16);
          if (bad_page) den = NAN;  // rows over a page that does not exist are NaN
          const int n = nt * 8 + (lane & 3) * 2 + j, item_row = first_row + n;
          if (item_row >= job.rows) continue;
          const int t = c.group_div.div(item_row);
          // a row that sees no key is zero; one whose visible scores are all -inf is 0 / 0
          const bool none = before + t < 0 && !bad_page;
          const float by = job.slot >= 0 ? 1.0f : 1.0f / den;
          T *const o = static_cast<T *>(c.out) + static_cast<int64_t>(job.t0 + t) * c.out_stride +
                       (static_cast<int64_t>(job.head) * c.group + (item_row - t * static_cast<int>(c.group))) * D;
          const size_t at = static_cast<size_t>(job.slot) * kRows + row0 + n;
#pragma unroll
          for (int md = 0; md < D / 16; md += 2) {
            const int d = md / (S::kBytes / 2) * 128 + lane / 4 * S::kBytes + md % (S::kBytes / 2) * 2;
            float x[4] = {acc[md][nt][j], acc[md][nt][2 + j], acc[md + 1][nt][j], acc[md + 1][nt][2 + j]};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = none ? 0.0f : x[e] * by;
            if (job.slot < 0) put4(o + d, x, c.out_wide);
            else *reinterpret_cast<float4 *>(c.part + at * D + d) = make_float4(x[0], x[1], x[2], x[3]);
          }
          if (job.slot >= 0 && lane < 4) c.part_ml[at] = make_float2(m[nt][j], den);
        }
      if (job.last >= 0 && rg == 0 && lane == 0)
        c.splits[sh.cta] = Split{job.slot, job.last, job.block * kRows, job.rows, job.t0, job.head * static_cast<int>(c.group), before};
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(ring.job_empty + slot * 8);
    if (++slot == P::slots) {
      slot = 0;
      job_phase ^= 1;
    }
  }
}

// ------------------------------------------------------------ host

// cuTensorMapEncodeTiled from the driver, looked up once through the runtime.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

std::atomic<unsigned> g_wait_clocks{kWaitClocks};

// Whether the cache's pages go by tensor copies: they hold whole groups of 8 keys, and the strides are not too long for
// them.  Boxes of 8 rows of 64 elements are 512 bytes: up to 8 rows per key head the copies' instructions take longer than
// asynchronous copies row by row; past that the shapes of 16 and 32 rows, which only boxes have, convert a code fewer times.  32
// requests up to 4096 keys, 8 key heads of 64, pages of 24, bf16, by boxes and by rows, at 3 / 8 / 9 / 16 / 17 / 32 rows per key
// head: 30.6 / 30.9 / 37.0 / 37.5 / 48.3 / 49.2 us and 27.2 / 27.5 / 42.7 / 42.9 / 59.4 / 75.7; f32: 31.4 / 31.7 / 42.0 / 43.3 /
// 62.1 / 64.0 and 27.7 / 28.0 / 44.5 / 45.1 / 62.3 / 80.2; pages of 8 and 40 alike.
bool takes_boxes(const gdn_attn_params &p) {
  const int64_t most = int64_t{1} << 40;
  return p.page_size % (p.head_dim == 64 && rows_of(p) <= 8 ? 16 : 8) == 0 && p.cache_page_stride < most && p.cache_head_stride < most && p.cache_slot_stride < most &&
         tensor_map_encoder() != nullptr;
}

// A cache as [head_dim, page_size, n_kv_heads, n_pages] with boxes of `rows` rows of 128 elements (or 64) within a page.
cudaError_t cache_map(CUtensorMap *map, const void *cache, const gdn_attn_params &p, uint32_t rows) {
  const cuuint64_t dims[4] = {p.head_dim, p.page_size, p.n_kv_heads, p.n_pages};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(p.cache_slot_stride), static_cast<cuuint64_t>(p.cache_head_stride),
                                 static_cast<cuuint64_t>(p.cache_page_stride)};
  const cuuint32_t box[4] = {p.head_dim < 128 ? p.head_dim : 128, rows, 1, 1}, step[4] = {1, 1, 1, 1};
  const CUresult r = tensor_map_encoder()(
      map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(cache), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
      p.head_dim < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Calls f with the variant of the call: the fewest rows per block that hold the rows of its requests.  A warp with two row
// tiles converts a code once for 16 rows, where two warps with one would do it twice (32 requests, windows of 1 to 4, 8 heads of
// 256 per key head: 71 us with four warps of a row tile each, 60 with two of two); q's fragments are in shared memory where they
// would not fit the registers.  32 requests up to 4096 keys, 8 key heads of 128, 12 rows: 54.6 us with six warps of 255
// registers, 47.9 with eight of 168; 32 rows: 69.8 and 75.6; of 64, 32 rows: 74.7 with one CTA, whose two feeding warps are too
// few, 46.2 with two.  f32, 12 rows, heads of 128: 65.4 us with six warps of 255 registers, 73.4 with eight of 168, which spill;
// of 64: 40.2 us with q's fragments in shared memory, 43.9 in registers.
template <typename F>
auto dispatch(const gdn_attn_params &p, bool boxed, F f) {
  const uint64_t rows = rows_of(p);
  auto by_dim = [&](auto t) {
    using T = decltype(t);
    constexpr bool f32 = sizeof(T) == 4;
    if (p.head_dim == 64)
      return !boxed       ? f(Pick8<T, 64, 1, 1, 4, 2, 2, 2, false>{})
             : rows <= 8  ? f(Pick8<T, 64, 1, 1, 4, 2, 2, 2, true>{})
             : rows <= 16 ? f(Pick8<T, 64, 2, 1, 4, 2, 2, 2, true, f32>{})
                          : f(Pick8<T, 64, 2, 2, 4, 2, 2, 2, true, f32>{});
    if (p.head_dim == 128)
      return !boxed       ? f(Pick8<T, 128, 1, 1, 4, 2, 2, 2, false, f32>{})
             : rows <= 8  ? f(Pick8<T, 128, 1, 1, 4, 2, 2, 2, true, f32>{})
             : rows <= 16 ? f(Pick8<T, 128, 2, 1, f32 ? 6 : 4, 2, f32 ? 2 : 1, f32 ? 1 : 2, true, true>{})
                          : f(Pick8<T, 128, 2, 2, 6, 2, 2, 1, true, true>{});
    return !boxed       ? f(Pick8<T, 256, 1, 1, 3, 1, 1, 2, false, f32>{})
           : rows <= 8  ? f(Pick8<T, 256, 1, 1, 3, 1, 1, 2, true, f32>{})
           : rows <= 16 ? f(Pick8<T, 256, 2, 1, 6, 2, 1, 1, true, true>{})
                        : f(Pick8<T, 256, 2, 2, 6, 2, 1, 1, true, true>{});
  };
  return p.dtype == GDN_DTYPE_BF16 ? by_dim(__nv_bfloat16{}) : by_dim(float{});
}

}  // namespace

// For either way of feeding: a call's pages and strides do not matter.
size_t attn_fp8_workspace_bytes(const gdn_attn_params &p) {
  auto bytes = [](auto pick) {
    using P = decltype(pick);
    return part_floats(P::ctas, P::rows, P::D) * 4 + static_cast<size_t>(2) * P::ctas * P::rows * sizeof(float2) +
           P::ctas * sizeof(Split);
  };
  const size_t boxed = dispatch(p, true, bytes), rows = dispatch(p, false, bytes);
  return boxed > rows ? boxed : rows;
}

cudaError_t launch_attn_paged_fp8(const AttnFp8Args &a, cudaStream_t stream) {
  const gdn_attn_params &p = a.p;
  Call c = call_of(p, a.q, a.k_cache, a.v_cache, a.block_table, a.kv_lens, a.token_start, a.output);
  c.k_scale = a.k_scale;
  c.v_scale = a.v_scale;
  c.wait_clocks = g_wait_clocks.load(std::memory_order_relaxed);
  c.q_wide = reinterpret_cast<uintptr_t>(a.q) % 16 == 0 && p.q_stride % (p.dtype == GDN_DTYPE_BF16 ? 8 : 4) == 0;
  return dispatch(p, takes_boxes(p), [&](auto pick) {
    using P = decltype(pick);
    using T = typename P::T;
    // boxes of 32, 16 or 8 rows, as divide a page
    CUtensorMap k_map = {}, v_map = {};
    if constexpr (P::BOXED) {
      c.box = p.page_size % 16 ? 8 : p.page_size % 32 || P::S::kTile == 16 ? 16 : 32;
      cudaError_t e = cache_map(&k_map, a.k_cache, p, c.box);
      if (e == cudaSuccess) e = cache_map(&v_map, a.v_cache, p, c.box);
      if (e != cudaSuccess) return e;
    }
    const uint64_t seen = static_cast<uint64_t>(p.window) + p.n_tokens;  // keys a window of tokens sees at most
    const uint64_t keys = static_cast<uint64_t>(p.max_pages) * p.page_size;
    c.whole_items = (p.window && seen < keys ? seen : keys) <= 256;
    c.splits = static_cast<Split *>(a.workspace);
    c.part = reinterpret_cast<float *>(c.splits + P::ctas);
    c.part_ml = reinterpret_cast<float2 *>(c.part + part_floats(P::ctas, P::rows, P::D));
    const auto main = gdn_attn_fp8_kernel<P>;
    cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, P::smem);
    if (e != cudaSuccess) return e;
    e = launch_in_order(main, dim3(P::ctas), P::threads, P::smem, stream, c, k_map, v_map);
    if (e != cudaSuccess || c.whole_items) return e;
    return launch_join<T, P::D, P::rows>(c, P::ctas, static_cast<uint64_t>(p.n_seqs) * p.n_kv_heads * 4 < P::ctas, stream);
  });
}

void attn_fp8_wait_clocks(uint32_t clocks) { g_wait_clocks.store(clocks ? clocks : kWaitClocks, std::memory_order_relaxed); }

cudaError_t attn_fp8_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
