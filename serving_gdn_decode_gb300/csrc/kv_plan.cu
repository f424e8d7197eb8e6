// The plan of one serving step over a paged key-value cache: block table, slot
// map, positions, lengths and token offsets from the request lengths.
//
// With need_s = max(owned_s, ceil((ctx_s + new_s) / page)) pages and
// demand_s = need_s - owned_s, exclusive prefix sums over the requests give
// each request's first new token (over new) and the rank of its first new page
// in the free stack (over demand).  Everything else is a lookup: token i of
// the step belongs to the last request that starts at or before it, stands at
// position ctx_s + i - start_s, and its page is the table's or, for a page new
// in this step, free_pages[n_free - 1 - rank].
//
// One launch and no waiting between CTAs: every CTA computes the same two
// prefix sums for itself, 256 or 1024 requests at a time, and writes its own share of
// the tokens, the new table entries and the per-request outputs.  Nothing a
// CTA reads is written by another (a table entry that exists before the call
// is only read, a new one only written; a new page's number comes from the
// free stack), so the inputs stay as they are and the outputs are new arrays.
//
// The data is a few KB to a few MB, so latency bounds it: one dependent load,
// a two-value scan over the CTA with one barrier, and the stores.  Measured on a
// GB300, back to back: 64 requests 3.3 us, 1024 requests with 58 prompts among
// them (32 thousand tokens) 5.6 us; a launch alone is about 2.
#include <cuda_runtime.h>

#include <climits>

#include "paged_common.cuh"
#include "paged_internal.h"

namespace gdn {
namespace {

constexpr uint32_t kTokensPerCta = 512;  // slots a CTA fills before another CTA is added
constexpr uint32_t kMaxCtas = 152;

struct Pair {
  long long tokens, pages;
};

__device__ __forceinline__ Pair warp_scan(Pair x, int lane) {  // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long t = __shfl_up_sync(0xffffffffu, x.tokens, d);
    const long long p = __shfl_up_sync(0xffffffffu, x.pages, d);
    if (lane >= d) {
      x.tokens += t;
      x.pages += p;
    }
  }
  return x;
}

// Exclusive prefix sums over the CTA's threads of x; *total: the sums over all.
// Every warp adds the warps' sums up for itself: one barrier.
template <int THREADS>
__device__ __forceinline__ Pair block_scan(Pair x, Pair *warp_sum /* THREADS / 32 in shared memory */, Pair *total) {
  constexpr int kWarps = THREADS / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Pair inc = warp_scan(x, lane);
  if (lane == 31) warp_sum[warp] = inc;
  __syncthreads();
  const Pair w = warp_scan(lane < kWarps ? warp_sum[lane] : Pair{0, 0}, lane);
  *total = Pair{__shfl_sync(0xffffffffu, w.tokens, kWarps - 1), __shfl_sync(0xffffffffu, w.pages, kWarps - 1)};
  Pair before{__shfl_sync(0xffffffffu, w.tokens, warp ? warp - 1 : 0), __shfl_sync(0xffffffffu, w.pages, warp ? warp - 1 : 0)};
  if (warp == 0) before = Pair{0, 0};
  return Pair{before.tokens + inc.tokens - x.tokens, before.pages + inc.pages - x.pages};
}

// Last of start[0..n) that is <= x (start[0] <= x, ascending, equal runs allowed).
__device__ __forceinline__ int last_at_or_before(const int *start, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int to_int(long long x) { return static_cast<int>(x < INT_MAX ? x : INT_MAX); }

template <int kThreads>
__global__ void __launch_bounds__(kThreads) gdn_kv_plan_kernel(const PlanArgs a, const FastDiv page_div) {
  __shared__ Pair warp_sum[32];
  __shared__ int s_start[kThreads], s_rank[kThreads], s_ctx[kThreads], s_owned[kThreads];
  __shared__ unsigned char s_served[kThreads];

  const gdn_kv_plan_params &p = a.p;
  const int tid = threadIdx.x;
  begin_in_order();
  const long long page = p.page_size;
  // this CTA's share of the slots
  const uint32_t per = (p.n_slots + gridDim.x - 1) / gridDim.x;
  const long long my0 = min(static_cast<long long>(blockIdx.x) * per, static_cast<long long>(p.n_slots));
  const long long my1 = min(my0 + per, static_cast<long long>(p.n_slots));

  unsigned int bad = 0;
  long long n_free = *a.n_free;
  if (n_free < 0 || n_free > p.n_free_max) {
    bad |= GDN_DEVICE_BAD_REQUEST;
    n_free = n_free < 0 ? 0 : p.n_free_max;
  }

  Pair carry{0, 0};
  long long used = 0;  // pages taken from the stack, as this thread's requests know
  for (uint32_t s0 = 0; s0 < p.n_seqs; s0 += kThreads) {
    const uint32_t s = s0 + tid;
    const int n_here = min(static_cast<uint32_t>(kThreads), p.n_seqs - s0);
    long long ctx = 0, fresh = 0, owned = 0;
    if (s < p.n_seqs) {
      ctx = a.ctx_lens[s];
      fresh = a.new_lens[s];
      owned = a.owned[s];
    }
    const bool wrong = ctx < 0 || fresh < 0 || owned < 0 || owned > p.max_pages || ctx > owned * page;
    if (fresh < 0) fresh = 0;
    long long need = wrong ? 0 : page_div.div(static_cast<uint32_t>(min(ctx + fresh + page - 1, static_cast<long long>(INT_MAX))));
    const bool fits = !wrong && need <= p.max_pages && ctx + fresh + page - 1 <= INT_MAX;
    need = need > owned ? need : owned;
    const long long demand = fits ? need - owned : 0;
    if (!fits) bad |= GDN_DEVICE_BAD_REQUEST;

    Pair total;
    Pair base = block_scan<kThreads>(Pair{fresh, demand}, warp_sum, &total);
    base.tokens += carry.tokens;
    base.pages += carry.pages;
    const bool served = fits && (demand == 0 || base.pages + demand <= n_free);
    if (fits && !served) bad |= GDN_DEVICE_OUT_OF_PAGES;
    if (served && demand > 0) used = base.pages + demand;
    s_start[tid] = to_int(base.tokens);
    s_rank[tid] = to_int(base.pages);
    s_ctx[tid] = static_cast<int>(wrong ? 0 : ctx);
    s_owned[tid] = static_cast<int>(owned);
    s_served[tid] = served;
    if (s < p.n_seqs && (s0 / kThreads) % gridDim.x == blockIdx.x) {
      a.kv_lens[s] = static_cast<int>(wrong ? 0 : served ? ctx + fresh : ctx);
      a.owned_out[s] = static_cast<int>(served ? need : owned);
      a.token_start[s] = to_int(base.tokens);
    }
    __syncthreads();

    // tokens of these requests in this CTA's share
    const long long t0 = max(my0, carry.tokens), t1 = min(my1, carry.tokens + total.tokens);
    for (long long i = t0 + tid; i < t1; i += kThreads) {
      const int r = last_at_or_before(s_start, n_here, static_cast<int>(i));
      const long long pos = static_cast<long long>(s_ctx[r]) + (i - s_start[r]);
      long long slot = -1;
      if (s_served[r]) {
        const uint32_t j = page_div.div(static_cast<uint32_t>(pos));
        const int pg = j < static_cast<uint32_t>(s_owned[r])
                           ? a.block_table[static_cast<uint64_t>(s0 + r) * p.max_pages + j]
                           : a.free_pages[n_free - 1 - (s_rank[r] + static_cast<long long>(j) - s_owned[r])];
        if (static_cast<uint32_t>(pg) < p.n_pages) slot = static_cast<long long>(pg) * page + (pos - j * page);
        else bad |= GDN_DEVICE_BAD_PAGE;
      }
      a.slot_map[i] = static_cast<int>(slot);
      a.positions[i] = to_int(pos);
    }
    // new table entries of these requests, by rank (ranks past the stack are never served)
    const long long ranks = min(total.pages, n_free - carry.pages);
    for (long long k = static_cast<long long>(blockIdx.x) * kThreads + tid; k < ranks;
         k += static_cast<long long>(gridDim.x) * kThreads) {
      const long long rank = carry.pages + k;
      const int r = last_at_or_before(s_rank, n_here, to_int(rank));
      if (s_served[r])
        a.block_table[static_cast<uint64_t>(s0 + r) * p.max_pages + s_owned[r] + (rank - s_rank[r])] =
            a.free_pages[n_free - 1 - rank];
    }
    carry.tokens += total.tokens;
    carry.pages += total.pages;
    __syncthreads();
  }

  // slots past the step's tokens
  for (long long i = max(my0, carry.tokens) + tid; i < my1; i += kThreads) {
    a.slot_map[i] = -1;
    a.positions[i] = 0;
  }
  if (carry.tokens > p.n_slots) bad |= GDN_DEVICE_BAD_REQUEST;
  if (blockIdx.x == 0) {
    // the served requests' pages are the first ranks of the stack
    Pair *most = warp_sum;
    long long m = used;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));
    if ((tid & 31) == 0) most[tid >> 5].pages = m;
    __syncthreads();
    if (tid == 0) {
      for (int w = 0; w < kThreads / 32; ++w) m = max(m, most[w].pages);
      *a.n_free_out = static_cast<int>(n_free - m);
      a.token_start[p.n_seqs] = to_int(carry.tokens);
    }
  }
  if (bad) report(bad);
}

}  // namespace

cudaError_t launch_kv_plan(const PlanArgs &a, cudaStream_t stream) {
  uint32_t ctas = (a.p.n_slots + kTokensPerCta - 1) / kTokensPerCta;
  if (ctas < 1) ctas = 1;
  if (ctas > kMaxCtas) ctas = kMaxCtas;
  // a CTA of the requests' number: the fewer warps, the sooner its barriers are passed
  const FastDiv page(a.p.page_size);
  if (a.p.n_seqs <= 256) return launch_in_order(gdn_kv_plan_kernel<256>, dim3(ctas), 256, 0, stream, a, page);
  return launch_in_order(gdn_kv_plan_kernel<1024>, dim3(ctas), 1024, 0, stream, a, page);
}

cudaError_t kv_plan_status_word(unsigned int **word) { return paged_status_word(word); }

}  // namespace gdn
