// C-ABI entry points of the full-attention operators: argument checks and
// dispatch (gdn_kv_plan, gdn_rope, gdn_rope_store, gdn_attn_paged).
#include <cuda_runtime.h>

#include <cmath>
#include <cstring>

#include "../../include/gdn.h"
#include "abi_common.h"
#include "paged_internal.h"

namespace {

using gdn::aligned;
using gdn::fail;
using gdn::Span;

// Slot numbers and key indices stay below this, so that a tile past the end
// still has 32-bit indices.
constexpr unsigned long long kMaxSlots = (1ull << 31) - (1ull << 16);

unsigned long long elem_bytes(uint32_t dtype) { return dtype == GDN_DTYPE_BF16 ? 2 : 4; }

// A buffer of `rows` rows of row_bytes, stride_bytes apart, at p.
struct Rows {
  const void *p;
  unsigned long long rows, row_bytes, stride_bytes;
  const char *name;
  Span span() const { return Span{p, rows ? (rows - 1) * stride_bytes + row_bytes : 0, name}; }
};

// Whether two buffers share a byte.  Views of one fused row (equal strides) lie
// within each other's span and are told apart by their place in the row.
bool rows_overlap(const Rows &a, const Rows &b) {
  if (a.rows == 0 || b.rows == 0 || !gdn::overlap(a.span(), b.span())) return false;
  if (a.stride_bytes == b.stride_bytes && a.stride_bytes > 0) {
    const unsigned long long s = a.stride_bytes;
    const unsigned long long pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const unsigned long long d = pb >= pa ? (pb - pa) % s : (s - (pa - pb) % s) % s;  // b's place after a's
    if (a.row_bytes <= d && d + b.row_bytes <= s) return false;
  }
  return true;
}

gdn_status cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return GDN_OK;
  return fail(GDN_ERR_CUDA, "gdn: kernel launch failed: %s", cudaGetErrorString(e));
}

gdn_status overlap_error(const Rows &a, const Rows &b) {
  return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s overlaps %s", a.name, b.name);
}

gdn_status check_ints(const Span &s) {
  if (s.bytes == 0) return GDN_OK;
  if (s.p == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s is NULL", s.name);
  if (!aligned(s.p, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s must be 4-byte aligned", s.name);
  return GDN_OK;
}

struct Cache {
  uint32_t n_pages, page_size, n_kv, dim;
  int64_t page_stride, head_stride, slot_stride;
  unsigned long long es;
};

// The sizes and strides alone, and the cache's extent.  What is only read may share rows.
gdn_status check_cache(const Cache &c, unsigned long long *bytes) {
  if (c.n_pages == 0 || c.page_size == 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: n_pages and page_size must be > 0");
  if (static_cast<unsigned long long>(c.n_pages) * c.page_size > kMaxSlots)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: n_pages x page_size must stay below 2^31 - 2^16");
  const int64_t most = int64_t{1} << 46;
  if (c.page_stride < c.dim || c.head_stride < c.dim || c.slot_stride < c.dim || c.page_stride > most ||
      c.head_stride > most || c.slot_stride > most)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: the cache strides must lie in [head_dim, 2^46]");
  const unsigned __int128 elems = static_cast<unsigned __int128>(c.n_pages - 1) * c.page_stride +
                                  static_cast<unsigned __int128>(c.n_kv - 1) * c.head_stride +
                                  static_cast<unsigned __int128>(c.page_size - 1) * c.slot_stride + c.dim;
  if (elems > (static_cast<unsigned __int128>(1) << 58))
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: the cache strides reach too far");
  *bytes = static_cast<unsigned long long>(elems) * c.es;
  return GDN_OK;
}

// What is stored into: each stride over an extent above 1 passes what the smaller ones cover, so that no two rows
// share an element.
class StoredCache {
 public:
  explicit StoredCache(const Cache &c) : row_(static_cast<int64_t>(c.dim * c.es)) {
    const struct { uint32_t extent; int64_t stride; } all[] = {
        {c.n_pages, c.page_stride}, {c.n_kv, c.head_stride}, {c.page_size, c.slot_stride}};
    for (const auto &x : all) {
      if (x.extent <= 1) continue;
      int i = n_++;
      for (; i > 0 && dims_[i - 1].stride < x.stride * static_cast<int64_t>(c.es); --i) dims_[i] = dims_[i - 1];
      dims_[i] = Dim{x.extent, x.stride * static_cast<int64_t>(c.es)};
    }
  }
  bool rows_apart() const {
    int64_t covered = row_;
    for (int i = n_ - 1; i >= 0; --i) {
      if (dims_[i].stride < covered) return false;
      covered += (dims_[i].extent - 1) * dims_[i].stride;
    }
    return true;
  }
  // Whether a cache of the same layout, `d` bytes on, shares a byte with this one (rows_apart() holds): whether d is
  // a difference of two places.  The smaller strides reach less far than the one at hand, so only the two multiples
  // of it on either side of d can be part of it.
  bool meets(int64_t d, int i = 0) const {
    if (i == n_) return -row_ < d && d < row_;
    const int64_t s = dims_[i].stride, below = d / s - (d % s < 0), most = dims_[i].extent - 1;
    for (int64_t x = below; x <= below + 1; ++x)
      if (-most <= x && x <= most && meets(d - x * s, i + 1)) return true;
    return false;
  }

 private:
  struct Dim { int64_t extent, stride; };  // in bytes, the largest first
  Dim dims_[3];
  int n_ = 0;
  int64_t row_;
};

gdn_status run_rope(const gdn::RopeArgs &x, bool store, const gdn_rope_params *params, gdn_stream_t stream) {
  gdn::g_last_error[0] = '\0';
  if (params == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: params is NULL");
  gdn::RopeArgs a = x;
  a.p = *params;
  const gdn_rope_params &p = a.p;
  if (p.dtype > GDN_DTYPE_BF16) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: unknown dtype %u", p.dtype);
  if (p.flags & ~(GDN_ROPE_INTERLEAVED | GDN_ROPE_INVERSE))
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: unknown rope flag bits 0x%x", p.flags);
  if (p.head_dim == 0 || p.head_dim > GDN_ROPE_MAX_DIM || p.head_dim % 2)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: head_dim (%u) must be even, at most %u", p.head_dim, GDN_ROPE_MAX_DIM);
  if (p.rot_dim == 0 || p.rot_dim > p.head_dim || p.rot_dim % 2)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: rot_dim (%u) must be even, in (0, head_dim]", p.rot_dim);
  if (p.n_q_heads == 0 || p.n_kv_heads == 0 || p.n_axes == 0 || p.n_positions == 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: heads, n_axes and n_positions must be > 0");
  if (p.n_q_heads > (1u << 20) || p.n_kv_heads > (1u << 20))
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: too many heads");
  if (p.n_tokens > 0x7fffffffu || p.n_positions > 0x7fffffffu)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: n_tokens and n_positions must be below 2^31");
  for (uint32_t j = 0; j < p.rot_dim / 2; ++j)
    if (p.axis_of_pair[j] >= p.n_axes)
      return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: axis_of_pair[%u] = %u, with %u axes", j, p.axis_of_pair[j], p.n_axes);
  if (store && (p.flags & GDN_ROPE_INVERSE))
    return fail(GDN_ERR_UNSUPPORTED, "gdn: gdn_rope_store has no inverse rotation");
  const unsigned long long es = elem_bytes(p.dtype), t = p.n_tokens;
  const unsigned long long qb = es * p.head_dim * p.n_q_heads, kb = es * p.head_dim * p.n_kv_heads;
  const struct { int64_t stride; unsigned long long row; const char *name; } st[] = {
      {p.q_stride, qb, "q_stride"}, {p.q_out_stride, qb, "q_out_stride"}, {p.k_stride, kb, "k_stride"},
      {store ? p.v_stride : p.k_out_stride, kb, store ? "v_stride" : "k_out_stride"}};
  for (const auto &s : st)
    if (s.stride < static_cast<int64_t>(s.row / es) || s.stride > (int64_t{1} << 40))
      return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s is shorter than a row, or above 2^40", s.name);
  if (p.positions_stride < 0 || p.positions_stride > (int64_t{1} << 40))
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: positions_stride must lie in [0, 2^40]");
  unsigned long long cache_bytes = 0;
  Cache cache{};
  if (store) {
    cache = Cache{p.n_pages, p.page_size, p.n_kv_heads, p.head_dim, p.cache_page_stride, p.cache_head_stride, p.cache_slot_stride, es};
    const gdn_status r = check_cache(cache, &cache_bytes);
    if (r != GDN_OK) return r;
  }
  const StoredCache stored(cache);
  if (store && !stored.rows_apart())
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: the cache strides let rows overlap");
  if (t == 0) return GDN_OK;
  const Rows in[] = {{a.q, t, qb, es * p.q_stride, "q"},
                     {a.k, t, kb, es * p.k_stride, "k"},
                     {a.positions, 1, 4 * ((p.n_axes - 1) * static_cast<unsigned long long>(p.positions_stride) + t), 0, "positions"},
                     {a.cos_sin, 1, 4ull * p.rot_dim * p.n_positions, 0, "cos_sin"},
                     {a.v, store ? t : 0, kb, es * p.v_stride, "v"},
                     {a.slot_map, store ? 1ull : 0ull, 4 * t, 0, "slot_map"}};
  const Rows cache_k{a.k_cache, 1, cache_bytes, 0, "k_cache"};
  const Rows rows_k{a.k_out, t, kb, es * p.k_out_stride, "k_out"};
  const Rows out[] = {{a.q_out, t, qb, es * p.q_out_stride, "q_out"},
                      store ? cache_k : rows_k,
                      {a.v_cache, store ? 1ull : 0ull, cache_bytes, 0, "v_cache"}};
  for (const Rows &b : in)
    if (b.rows && b.p == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s is NULL", b.name);
  for (const Rows &b : out)
    if (b.rows && b.p == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s is NULL", b.name);
  const Rows *ints[] = {&in[2], &in[3], &in[5]};
  for (const Rows *b : ints)
    if (b->rows && !aligned(b->p, 4)) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s must be 4-byte aligned", b->name);
  const Rows *data[] = {&in[0], &in[1], &in[4], &out[0], &out[1], &out[2]};
  for (const Rows *b : data)
    if (b->rows && !aligned(b->p, es))
      return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s must be aligned to an element", b->name);
  for (int o = 0; o < 3; ++o) {
    for (int i = 0; i < 6; ++i) {
      // q_out may be q, k_out may be k: a thread reads what it overwrites
      if (o == i && (o == 0 || (o == 1 && !store)) && out[o].p == in[i].p && out[o].stride_bytes == in[i].stride_bytes)
        continue;
      if (rows_overlap(out[o], in[i])) return overlap_error(out[o], in[i]);
    }
    for (int i = 0; i < o; ++i) {
      // k_cache and v_cache may be two views of one array: pages of K and V in turn, or heads, or slots
      if (o == 2 && i == 1) {
        if (store && stored.meets(static_cast<int64_t>(reinterpret_cast<uintptr_t>(out[o].p) - reinterpret_cast<uintptr_t>(out[i].p))))
          return overlap_error(out[o], out[i]);
        continue;
      }
      if (rows_overlap(out[o], out[i])) return overlap_error(out[o], out[i]);
    }
  }
  return cuda_status(gdn::launch_rope(a, reinterpret_cast<cudaStream_t>(stream)));
}

// The checks of a gdn_attn_params block alone.
gdn_status check_attn_params(const gdn_attn_params *params, unsigned long long *cache_bytes) {
  if (params == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: params is NULL");
  const gdn_attn_params &p = *params;
  if (p.dtype > GDN_DTYPE_BF16) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: unknown dtype %u", p.dtype);
  if (p.n_q_heads == 0 || p.n_kv_heads == 0 || p.n_seqs == 0 || p.max_pages == 0 || p.head_dim == 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: heads, head_dim, n_seqs and max_pages must be > 0");
  if (p.n_q_heads % p.n_kv_heads)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: n_q_heads (%u) must be a multiple of n_kv_heads (%u)", p.n_q_heads,
                p.n_kv_heads);
  if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256)
    return fail(GDN_ERR_UNSUPPORTED, "gdn: head_dim %u has no attention kernel; use 64, 128 or 256", p.head_dim);
  if (static_cast<unsigned long long>(p.n_tokens) * p.n_q_heads > 0x7fff0000ull || p.n_seqs > 0x7fff0000u)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: n_seqs and n_tokens x n_q_heads must stay below 2^31 - 2^16");
  if (!std::isfinite(p.scale)) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: scale must be finite");
  const unsigned long long es = elem_bytes(p.dtype);
  const gdn_status r = check_cache(Cache{p.n_pages, p.page_size, p.n_kv_heads, p.head_dim, p.cache_page_stride,
                                         p.cache_head_stride, p.cache_slot_stride, es}, cache_bytes);
  if (r != GDN_OK) return r;
  if (static_cast<unsigned long long>(p.max_pages) * p.page_size > kMaxSlots)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: max_pages x page_size must stay below 2^31 - 2^16");
  const int64_t e16 = 16 / static_cast<int64_t>(es);
  if (p.cache_page_stride % e16 || p.cache_head_stride % e16 || p.cache_slot_stride % e16)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: the cache strides must be multiples of 16 bytes");
  const int64_t row = static_cast<int64_t>(p.head_dim) * p.n_q_heads;
  if (p.q_stride < row || p.out_stride < row || p.q_stride > (int64_t{1} << 40) || p.out_stride > (int64_t{1} << 40))
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: q_stride or out_stride is shorter than a row, or above 2^40");
  if (p.dtype == GDN_DTYPE_BF16 && p.q_stride % 2)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: q_stride must be even in bf16");
  return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *owned,
                       const int32_t *free_pages, const int32_t *n_free, int32_t *block_table,
                       int32_t *kv_lens, int32_t *owned_out, int32_t *n_free_out,
                       int32_t *token_start, int32_t *slot_map, int32_t *positions,
                       const gdn_kv_plan_params *params, gdn_stream_t stream) {
  gdn::g_last_error[0] = '\0';
  if (params == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: params is NULL");
  const gdn_kv_plan_params &p = *params;
  if (p.n_seqs == 0 || p.page_size == 0 || p.n_pages == 0 || p.max_pages == 0)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: n_seqs, page_size, n_pages and max_pages must be > 0");
  if (static_cast<unsigned long long>(p.n_pages) * p.page_size > kMaxSlots ||
      static_cast<unsigned long long>(p.max_pages) * p.page_size > kMaxSlots || p.n_slots > kMaxSlots ||
      p.n_seqs > kMaxSlots || p.n_free_max > kMaxSlots)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: page counts x page_size, n_seqs, n_slots and n_free_max must stay below 2^31 - 2^16");
  const unsigned long long n = p.n_seqs;
  const Span in[] = {{ctx_lens, 4 * n, "ctx_lens"}, {new_lens, 4 * n, "new_lens"}, {owned, 4 * n, "owned"},
                     {free_pages, 4ull * p.n_free_max, "free_pages"}, {n_free, 4, "n_free"}};
  const Span out[] = {{block_table, 4 * n * p.max_pages, "block_table"}, {kv_lens, 4 * n, "kv_lens"},
                      {owned_out, 4 * n, "owned_out"}, {n_free_out, 4, "n_free_out"},
                      {token_start, 4 * (n + 1), "token_start"}, {slot_map, 4ull * p.n_slots, "slot_map"},
                      {positions, 4ull * p.n_slots, "positions"}};
  for (const Span &s : in)
    if (check_ints(s) != GDN_OK) return GDN_ERR_INVALID_ARGUMENT;
  for (const Span &s : out)
    if (check_ints(s) != GDN_OK) return GDN_ERR_INVALID_ARGUMENT;
  for (size_t o = 0; o < sizeof out / sizeof out[0]; ++o) {
    if (out[o].bytes == 0) continue;
    for (const Span &s : in)
      if (s.bytes && gdn::overlap(out[o], s))
        return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s overlaps %s", out[o].name, s.name);
    for (size_t i = 0; i < o; ++i)
      if (out[i].bytes && gdn::overlap(out[o], out[i]))
        return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s overlaps %s", out[o].name, out[i].name);
  }
  const gdn::PlanArgs a{ctx_lens, new_lens, owned, free_pages, n_free, block_table, kv_lens,
                        owned_out, n_free_out, token_start, slot_map, positions, p};
  return cuda_status(gdn::launch_kv_plan(a, reinterpret_cast<cudaStream_t>(stream)));
}

gdn_status gdn_rope(const void *q, const void *k, const int32_t *positions, const float *cos_sin,
                    void *q_out, void *k_out, const gdn_rope_params *params, gdn_stream_t stream) {
  gdn::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.q_out = q_out;
  a.k_out = k_out;
  return run_rope(a, false, params, stream);
}

gdn_status gdn_rope_store(const void *q, const void *k, const void *v, const int32_t *positions,
                          const float *cos_sin, const int32_t *slot_map, void *q_out, void *k_cache,
                          void *v_cache, const gdn_rope_params *params, gdn_stream_t stream) {
  gdn::RopeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.positions = positions;
  a.cos_sin = cos_sin;
  a.slot_map = slot_map;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  return run_rope(a, true, params, stream);
}

gdn_status gdn_attn_workspace_size(const gdn_attn_params *params, size_t *bytes) {
  gdn::g_last_error[0] = '\0';
  if (bytes == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: bytes is NULL");
  *bytes = 0;
  unsigned long long cache_bytes;
  const gdn_status r = check_attn_params(params, &cache_bytes);
  if (r != GDN_OK) return r;
  *bytes = gdn::attn_workspace_bytes(*params);
  return GDN_OK;
}

gdn_status gdn_attn_paged(const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *kv_lens,
                          const int32_t *token_start, void *output, const gdn_attn_params *params,
                          void *workspace, size_t workspace_bytes, gdn_stream_t stream) {
  gdn::g_last_error[0] = '\0';
  unsigned long long cache_bytes = 0;
  const gdn_status r = check_attn_params(params, &cache_bytes);
  if (r != GDN_OK) return r;
  const gdn_attn_params &p = *params;
  if (token_start == nullptr && p.n_tokens < p.n_seqs)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: without token_start q needs a row per request (%u rows, %u requests)",
                p.n_tokens, p.n_seqs);
  if (p.n_tokens == 0) return GDN_OK;
  const unsigned long long es = elem_bytes(p.dtype), row = es * p.head_dim * p.n_q_heads;
  const size_t need = gdn::attn_workspace_bytes(p);
  const Rows in[] = {{q, p.n_tokens, row, es * p.q_stride, "q"},
                     {k_cache, 1, cache_bytes, 0, "k_cache"},
                     {v_cache, 1, cache_bytes, 0, "v_cache"},
                     {block_table, 1, 4ull * p.n_seqs * p.max_pages, 0, "block_table"},
                     {kv_lens, 1, 4ull * p.n_seqs, 0, "kv_lens"},
                     {token_start, token_start ? 1ull : 0ull, 4ull * (p.n_seqs + 1ull), 0, "token_start"}};
  const Rows out{output, p.n_tokens, row, es * p.out_stride, "output"};
  const Rows ws{workspace, 1, need, 0, "workspace"};
  for (const Rows &b : in)
    if (b.rows && b.p == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s is NULL", b.name);
  if (output == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: output is NULL");
  if (workspace == nullptr) return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: workspace is NULL");
  if (workspace_bytes < need)
    return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: workspace has %zu bytes, %zu needed", workspace_bytes, need);
  const struct { const void *p; uintptr_t a; const char *name; } al[] = {
      {q, 4, "q"},           {k_cache, 16, "k_cache"}, {v_cache, 16, "v_cache"}, {block_table, 4, "block_table"},
      {kv_lens, 4, "kv_lens"}, {token_start, 4, "token_start"}, {output, es, "output"}, {workspace, 16, "workspace"}};
  for (const auto &x : al)
    if (!aligned(x.p, x.a))
      return fail(GDN_ERR_INVALID_ARGUMENT, "gdn: %s must be %u-byte aligned", x.name, static_cast<unsigned>(x.a));
  for (const Rows &b : in) {
    if (rows_overlap(out, b)) return overlap_error(out, b);
    if (rows_overlap(ws, b)) return overlap_error(ws, b);
  }
  if (rows_overlap(ws, out)) return overlap_error(ws, out);
  gdn::AttnArgs a{q, k_cache, v_cache, block_table, kv_lens, token_start, output, p, workspace};
  return cuda_status(gdn::launch_attn_paged(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
