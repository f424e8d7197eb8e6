// Python binding of the full-attention operators over torch tensors (module
// _paged_binding, wrapped by paged.py).  Argument marshalling only: a tensor's
// shape, strides, type and address become the params and pointers of the C ABI
// call, which checks the rest.  Compiled, because a decode step makes these
// calls for every layer: reading a tensor's attributes from Python would take
// longer than the kernels.
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "../../include/gdn.h"

namespace {

PyObject *g_error = nullptr;  // GdnError(status, message)

// Sets GdnError; always false.
bool fail(int status, const char *fmt, ...) {
  char msg[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof msg, fmt, ap);
  va_end(ap);
  PyObject *args = Py_BuildValue("(is)", status, msg);
  PyObject *e = args ? PyObject_CallObject(g_error, args) : nullptr;
  if (e) PyErr_SetObject(g_error, e);
  Py_XDECREF(e);
  Py_XDECREF(args);
  return false;
}
bool bad(const char *name, const char *what) { return fail(GDN_ERR_INVALID_ARGUMENT, "%s %s", name, what); }

PyObject *finish(gdn_status st) {
  if (st == GDN_OK) Py_RETURN_NONE;
  fail(st, "%s", gdn_last_error());
  return nullptr;
}

struct Arg {
  const char *name;
  const at::Tensor *t;
  const at::Tensor *operator->() const { return t; }
  void *ptr() const { return t->data_ptr(); }
};

bool get(PyObject *o, const char *name, Arg *out) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s must be a torch.Tensor (got %s)", name, Py_TYPE(o)->tp_name);
    return false;
  }
  *out = Arg{name, &THPVariable_Unpack(o)};
  return true;
}

const char *name_of(at::ScalarType t) { return t == at::kBFloat16 ? "bf16" : t == at::kFloat ? "f32" : t == at::kInt ? "int32" : t == at::kFloat8_e4m3fn ? "e4m3" : "another type"; }

bool want_type(const Arg &a, at::ScalarType t) {
  if (a->scalar_type() == t) return true;
  return fail(GDN_ERR_INVALID_ARGUMENT, "%s must be %s (got %s)", a.name, name_of(t), c10::toString(a->scalar_type()));
}

// int32, contiguous, of n elements (rows x n when rows >= 0)
bool want_ints(const Arg &a, int64_t n, int64_t rows = -1) {
  if (!want_type(a, at::kInt)) return false;
  const bool shape = rows < 0 ? a->dim() == 1 && a->size(0) == n : a->dim() == 2 && a->size(0) == rows && a->size(1) == n;
  if (shape && a->is_contiguous()) return true;
  return rows < 0 ? fail(GDN_ERR_INVALID_ARGUMENT, "%s must be contiguous, of %lld elements", a.name, static_cast<long long>(n))
                  : fail(GDN_ERR_INVALID_ARGUMENT, "%s must be contiguous, of %lld x %lld elements", a.name,
                         static_cast<long long>(rows), static_cast<long long>(n));
}

bool data_type(const Arg &a, uint32_t *dtype) {
  if (a->scalar_type() == at::kFloat) *dtype = GDN_DTYPE_F32;
  else if (a->scalar_type() == at::kBFloat16) *dtype = GDN_DTYPE_BF16;
  else return bad(a.name, "must be f32 or bf16");
  return true;
}

// [n_tokens, n_heads, head_dim] with contiguous rows; the token stride
bool want_rows(const Arg &a, at::ScalarType t, int64_t n, int64_t heads, int64_t dim, int64_t *stride) {
  if (!want_type(a, t)) return false;
  if (a->dim() != 3 || a->size(0) != n || a->size(1) != heads || a->size(2) != dim)
    return fail(GDN_ERR_INVALID_ARGUMENT, "%s must have shape [%lld, %lld, %lld]", a.name, static_cast<long long>(n),
                static_cast<long long>(heads), static_cast<long long>(dim));
  if ((dim > 1 && a->stride(2) != 1) || (heads > 1 && a->stride(1) != dim))
    return bad(a.name, "must have the heads of a token contiguous");
  *stride = n > 1 ? a->stride(0) : heads * dim;
  return true;
}

// [n_pages, n_kv_heads, page_size, head_dim], both of one layout; a stride of a
// dimension of size 1 says nothing and is given a harmless value
template <typename P>
bool want_cache(const Arg &k, const Arg &v, at::ScalarType t, int64_t dim, P *p, uint32_t *n_kv) {
  if (!want_type(k, t) || !want_type(v, t)) return false;
  bool one_layout = k->dim() == 4 && k->sizes() == v->sizes();
  for (int i = 0; one_layout && i < 4; ++i) one_layout = k->size(i) <= 1 || k->stride(i) == v->stride(i);
  if (!one_layout)
    return fail(GDN_ERR_INVALID_ARGUMENT,
                "k_cache and v_cache must be [n_pages, n_kv_heads, page_size, head_dim] of one layout");
  if (k->size(3) != dim || (*n_kv && k->size(1) != *n_kv))
    return fail(GDN_ERR_INVALID_ARGUMENT, "k_cache has %lld heads of %lld, expected %lld of %lld", static_cast<long long>(k->size(1)),
                static_cast<long long>(k->size(3)), static_cast<long long>(*n_kv ? *n_kv : k->size(1)), static_cast<long long>(dim));
  if (dim > 1 && k->stride(3) != 1) return bad("k_cache", "must have contiguous rows of head_dim");
  int64_t s[3], most = dim;
  for (int i = 0; i < 3; ++i) {
    s[i] = k->stride(i);
    if (k->size(i) > 1 && s[i] > most) most = s[i];
  }
  for (int i = 0; i < 3; ++i)
    if (k->size(i) <= 1) s[i] = most;
  p->n_pages = static_cast<uint32_t>(k->size(0));
  *n_kv = static_cast<uint32_t>(k->size(1));
  p->page_size = static_cast<uint32_t>(k->size(2));
  p->cache_page_stride = s[0];
  p->cache_head_stride = s[1];
  p->cache_slot_stride = s[2];
  return true;
}

// Sizes are 32-bit in the C ABI.
bool small(const Arg &a) {
  for (int64_t n : a->sizes())
    if (n > INT32_MAX) return bad(a.name, "has a dimension of 2^31 or more");
  return true;
}

bool on_one_device(const Arg *args, int n) {
  for (int i = 0; i < n; ++i) {
    if (!args[i]->is_cuda()) return bad(args[i].name, "must be a CUDA tensor");
    if (args[i]->get_device() != args[0]->get_device()) {
      char what[96];
      std::snprintf(what, sizeof what, "must be on %s's device", args[0].name);
      return bad(args[i].name, what);
    }
  }
  return true;
}

bool get_stream(PyObject *o, c10::DeviceIndex device, gdn_stream_t *out) {
  if (o == Py_None) {
    *out = reinterpret_cast<gdn_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
    return true;
  }
  PyObject *handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!handle) return false;
  void *p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (!p && PyErr_Occurred()) return false;
  *out = static_cast<gdn_stream_t>(p);
  return true;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

bool get_u32(PyObject *o, const char *name, uint32_t *out) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) return false;
  if (x < 0 || x > UINT32_MAX) return bad(name, "must lie in [0, 2^32)");
  *out = static_cast<uint32_t>(x);
  return true;
}

// ------------------------------------------------------------------ plan

// kv_plan(12 tensors in the C call's order, page_size, n_pages, stream)
PyObject *py_kv_plan(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  static const char *const names[12] = {"ctx_lens", "new_lens", "owned", "free_pages", "n_free", "block_table", "kv_lens",
                                        "owned_out", "n_free_out", "token_start", "slot_map", "positions"};
  if (!count(n_args, 15)) return nullptr;
  Arg a[12];
  for (int i = 0; i < 12; ++i)
    if (!get(args[i], names[i], &a[i]) || !small(a[i])) return nullptr;
  gdn_kv_plan_params p{};
  if (!get_u32(args[12], "page_size", &p.page_size) || !get_u32(args[13], "n_pages", &p.n_pages)) return nullptr;
  const int64_t n = a[0]->numel();
  if (a[5]->dim() != 2) {
    bad("block_table", "must be [n_seqs, max_pages]");
    return nullptr;
  }
  const int64_t slots = a[10]->numel();
  const int64_t sizes[12] = {n, n, n, a[3]->numel(), 1, a[5]->size(1), n, n, 1, n + 1, slots, slots};
  for (int i = 0; i < 12; ++i)
    if (!want_ints(a[i], sizes[i], i == 5 ? n : -1)) return nullptr;
  if (!on_one_device(a, 12)) return nullptr;
  p.n_seqs = static_cast<uint32_t>(n);
  p.max_pages = static_cast<uint32_t>(sizes[5]);
  p.n_free_max = static_cast<uint32_t>(sizes[3]);
  p.n_slots = static_cast<uint32_t>(slots);
  gdn_stream_t stream;
  if (!get_stream(args[14], a[0]->get_device(), &stream)) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a[0]->get_device()));
  auto in = [&](int i) { return static_cast<const int32_t *>(a[i].ptr()); };
  auto out = [&](int i) { return static_cast<int32_t *>(a[i].ptr()); };
  return finish(gdn_kv_plan(in(0), in(1), in(2), in(3), in(4), out(5), out(6), out(7), out(8), out(9), out(10), out(11), &p, stream));
}

// ------------------------------------------------------------------ rope

// The part of the params that gdn_rope and gdn_rope_store share.
bool rope_params(const Arg &q, const Arg &k, const Arg &positions, const Arg &cos_sin, const Arg &q_out, PyObject *axes,
                 gdn_rope_params *p) {
  if (!data_type(q, &p->dtype)) return false;
  if (q->dim() != 3 || k->dim() != 3) return bad(q->dim() != 3 ? "q" : "k", "must be [n_tokens, n_heads, head_dim]");
  const int64_t n = q->size(0), dim = q->size(2);
  p->head_dim = static_cast<uint32_t>(dim);
  p->n_tokens = static_cast<uint32_t>(n);
  p->n_q_heads = static_cast<uint32_t>(q->size(1));
  p->n_kv_heads = static_cast<uint32_t>(k->size(1));
  const at::ScalarType t = q->scalar_type();
  if (!want_rows(q, t, n, q->size(1), dim, &p->q_stride) || !want_rows(k, t, n, k->size(1), dim, &p->k_stride) ||
      !want_rows(q_out, t, n, q->size(1), dim, &p->q_out_stride))
    return false;
  const int64_t pd = positions->dim();
  if (positions->scalar_type() != at::kInt || pd < 1 || pd > 2 || positions->size(pd - 1) != n ||
      (n > 1 && positions->stride(pd - 1) != 1))
    return bad("positions", "must be int32 [n_tokens] or [n_axes, n_tokens] with contiguous rows");
  p->n_axes = pd == 2 ? static_cast<uint32_t>(positions->size(0)) : 1;
  p->positions_stride = pd == 2 && p->n_axes > 1 ? positions->stride(0) : 0;
  if (cos_sin->scalar_type() != at::kFloat || cos_sin->dim() != 2 || !cos_sin->is_contiguous())
    return bad("cos_sin", "must be contiguous f32 [n_positions, rot_dim]");
  p->n_positions = static_cast<uint32_t>(cos_sin->size(0));
  p->rot_dim = static_cast<uint32_t>(cos_sin->size(1));
  if (axes != Py_None) {
    char *bytes;
    Py_ssize_t len;
    if (PyBytes_AsStringAndSize(axes, &bytes, &len) < 0) return false;
    if (len != static_cast<Py_ssize_t>(p->rot_dim / 2))
      return fail(GDN_ERR_INVALID_ARGUMENT, "axes has %zd entries, expected rot_dim / 2 = %u", len, p->rot_dim / 2);
    if (p->rot_dim <= GDN_ROPE_MAX_DIM) memcpy(p->axis_of_pair, bytes, static_cast<size_t>(len));
  }
  return true;
}

// rope(q, k, positions, cos_sin, q_out, k_out, axes, flags, stream)
PyObject *py_rope(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  static const char *const names[6] = {"q", "k", "positions", "cos_sin", "q_out", "k_out"};
  if (!count(n_args, 9)) return nullptr;
  Arg a[6];
  for (int i = 0; i < 6; ++i)
    if (!get(args[i], names[i], &a[i]) || !small(a[i])) return nullptr;
  gdn_rope_params p{};
  if (!get_u32(args[7], "flags", &p.flags) || !rope_params(a[0], a[1], a[2], a[3], a[4], args[6], &p) ||
      !want_rows(a[5], a[0]->scalar_type(), p.n_tokens, p.n_kv_heads, p.head_dim, &p.k_out_stride) || !on_one_device(a, 6))
    return nullptr;
  gdn_stream_t stream;
  if (!get_stream(args[8], a[0]->get_device(), &stream)) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a[0]->get_device()));
  return finish(gdn_rope(a[0].ptr(), a[1].ptr(), static_cast<const int32_t *>(a[2].ptr()), static_cast<const float *>(a[3].ptr()),
                         a[4].ptr(), a[5].ptr(), &p, stream));
}

// rope_store(q, k, v, positions, cos_sin, slot_map, q_out, k_cache, v_cache, axes, flags, stream)
PyObject *py_rope_store(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  static const char *const names[9] = {"q", "k", "v", "positions", "cos_sin", "slot_map", "q_out", "k_cache", "v_cache"};
  if (!count(n_args, 12)) return nullptr;
  Arg a[9];
  for (int i = 0; i < 9; ++i)
    if (!get(args[i], names[i], &a[i]) || !small(a[i])) return nullptr;
  gdn_rope_params p{};
  if (!get_u32(args[10], "flags", &p.flags) || !rope_params(a[0], a[1], a[3], a[4], a[6], args[9], &p)) return nullptr;
  const at::ScalarType t = a[0]->scalar_type();
  uint32_t n_kv = p.n_kv_heads;
  if (!want_rows(a[2], t, p.n_tokens, p.n_kv_heads, p.head_dim, &p.v_stride) || !want_ints(a[5], p.n_tokens) ||
      !want_cache(a[7], a[8], t, p.head_dim, &p, &n_kv) || !on_one_device(a, 9))
    return nullptr;
  gdn_stream_t stream;
  if (!get_stream(args[11], a[0]->get_device(), &stream)) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a[0]->get_device()));
  return finish(gdn_rope_store(a[0].ptr(), a[1].ptr(), a[2].ptr(), static_cast<const int32_t *>(a[3].ptr()),
                               static_cast<const float *>(a[4].ptr()), static_cast<const int32_t *>(a[5].ptr()), a[6].ptr(),
                               a[7].ptr(), a[8].ptr(), &p, stream));
}

// ------------------------------------------------------------------ attention

bool attn_params(const Arg &q, const Arg &k, const Arg &v, bool fp8, gdn_attn_params *p) {
  if (!data_type(q, &p->dtype)) return false;
  if (q->dim() != 3) return bad("q", "must be [n_tokens, n_q_heads, head_dim]");
  p->n_tokens = static_cast<uint32_t>(q->size(0));
  p->n_q_heads = static_cast<uint32_t>(q->size(1));
  p->head_dim = static_cast<uint32_t>(q->size(2));
  p->n_kv_heads = 0;
  return want_rows(q, q->scalar_type(), q->size(0), q->size(1), q->size(2), &p->q_stride) &&
         want_cache(k, v, fp8 ? at::kFloat8_e4m3fn : q->scalar_type(), q->size(2), p, &p->n_kv_heads);
}

// f32 [n_pages, n_kv_heads], contiguous
bool want_scales(const Arg &a, int64_t n_pages, int64_t n_kv) {
  if (!want_type(a, at::kFloat)) return false;
  if (a->dim() == 2 && a->size(0) == n_pages && a->size(1) == n_kv && a->is_contiguous()) return true;
  return fail(GDN_ERR_INVALID_ARGUMENT, "%s must be contiguous, of %lld x %lld elements", a.name, static_cast<long long>(n_pages),
              static_cast<long long>(n_kv));
}

// attn_workspace_size(q, k_cache, n_seqs), attn_fp8_workspace_size(q, k_cache, n_seqs)
template <bool FP8>
PyObject *py_attn_workspace_size(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  if (!count(n_args, 3)) return nullptr;
  Arg q, k;
  gdn_attn_params p{};
  if (!get(args[0], "q", &q) || !get(args[1], "k_cache", &k) || !small(q) || !small(k) || !get_u32(args[2], "n_seqs", &p.n_seqs) ||
      !attn_params(q, k, k, FP8, &p))
    return nullptr;
  p.max_pages = 1;
  p.scale = 1.0f;
  p.out_stride = static_cast<int64_t>(p.n_q_heads) * p.head_dim;
  size_t bytes = 0;
  const gdn_status st = FP8 ? gdn_attn_fp8_workspace_size(&p, &bytes) : gdn_attn_workspace_size(&p, &bytes);
  if (st != GDN_OK) return finish(st);
  return PyLong_FromSize_t(bytes);
}

// attn_paged(q, k_cache, v_cache, block_table, kv_lens, token_start | None, output, workspace, scale | None, window, stream),
// attn_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, ...)
template <bool FP8>
PyObject *py_attn_paged(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  static const char *const names[10] = {"q", "k_cache", "v_cache", "block_table", "kv_lens", "token_start", "output", "workspace",
                                        "k_scale", "v_scale"};
  constexpr int kArgs = FP8 ? 10 : 8;
  if (!count(n_args, kArgs + 3)) return nullptr;
  // the scales, where there are any, stand behind the caches in the call and last here
  auto place = [](int i) { return !FP8 || i < 3 ? i : i < 8 ? i + 2 : i - 5; };
  PyObject *const *const more = args + kArgs;  // scale, window, stream
  const bool ragged = args[place(5)] != Py_None;
  Arg a[kArgs];
  for (int i = 0; i < kArgs; ++i) {
    if (i == 5 && !ragged) a[i] = a[4];
    else if (!get(args[place(i)], names[i], &a[i]) || (i != 7 && !small(a[i]))) return nullptr;
  }
  gdn_attn_params p{};
  if (!attn_params(a[0], a[1], a[2], FP8, &p) || !get_u32(more[1], "window", &p.window)) return nullptr;
  const int64_t n = a[4]->numel();
  if (a[3]->dim() != 2) {
    bad("block_table", "must be [n_seqs, max_pages]");
    return nullptr;
  }
  if (!want_ints(a[3], a[3]->size(1), n) || !want_ints(a[4], n) || (ragged && !want_ints(a[5], n + 1)) ||
      !want_rows(a[6], a[0]->scalar_type(), p.n_tokens, p.n_q_heads, p.head_dim, &p.out_stride))
    return nullptr;
  if constexpr (FP8)
    if (!want_scales(a[8], p.n_pages, p.n_kv_heads) || !want_scales(a[9], p.n_pages, p.n_kv_heads)) return nullptr;
  if (!a[7]->is_contiguous()) {
    bad("workspace", "must be contiguous");
    return nullptr;
  }
  if (!on_one_device(a, kArgs)) return nullptr;
  p.n_seqs = static_cast<uint32_t>(n);
  p.max_pages = static_cast<uint32_t>(a[3]->size(1));
  if (more[0] == Py_None) {
    p.scale = static_cast<float>(1.0 / std::sqrt(static_cast<double>(p.head_dim)));
  } else {
    const double s = PyFloat_AsDouble(more[0]);
    if (s == -1.0 && PyErr_Occurred()) return nullptr;
    p.scale = static_cast<float>(s);
  }
  gdn_stream_t stream;
  if (!get_stream(more[2], a[0]->get_device(), &stream)) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a[0]->get_device()));
  const int32_t *table = static_cast<const int32_t *>(a[3].ptr()), *lens = static_cast<const int32_t *>(a[4].ptr()),
                *start = ragged ? static_cast<const int32_t *>(a[5].ptr()) : nullptr;
  const size_t bytes = static_cast<size_t>(a[7]->nbytes());
  if constexpr (FP8)
    return finish(gdn_attn_paged_fp8(a[0].ptr(), a[1].ptr(), a[2].ptr(), static_cast<const float *>(a[8].ptr()),
                                     static_cast<const float *>(a[9].ptr()), table, lens, start, a[6].ptr(), &p, a[7].ptr(), bytes, stream));
  else
    return finish(gdn_attn_paged(a[0].ptr(), a[1].ptr(), a[2].ptr(), table, lens, start, a[6].ptr(), &p, a[7].ptr(), bytes, stream));
}

// ------------------------------------------------------------------ the 8-bit cache

// kv_store_fp8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream),
// kv_load_fp8(slot_map, k_cache, v_cache, k_scale, v_scale, k, v, stream)
template <bool STORE>
PyObject *py_kv_fp8(PyObject *, PyObject *const *args, Py_ssize_t n_args) {
  static const char *const names[7] = {"k", "v", "slot_map", "k_cache", "v_cache", "k_scale", "v_scale"};
  if (!count(n_args, 8)) return nullptr;
  Arg a[7];
  for (int i = 0; i < 7; ++i)
    if (!get(args[STORE ? i : (i + 5) % 7], names[i], &a[i]) || !small(a[i])) return nullptr;
  gdn_kv_fp8_params p{};
  if (!data_type(a[0], &p.dtype)) return nullptr;
  if (a[0]->dim() != 3) {
    bad("k", "must be [n_tokens, n_kv_heads, head_dim]");
    return nullptr;
  }
  const at::ScalarType t = a[0]->scalar_type();
  const int64_t n = a[0]->size(0), heads = a[0]->size(1), dim = a[0]->size(2);
  uint32_t n_kv = static_cast<uint32_t>(heads);
  if (!want_rows(a[0], t, n, heads, dim, &p.k_stride) || !want_rows(a[1], t, n, heads, dim, &p.v_stride) || !want_ints(a[2], n) ||
      !want_cache(a[3], a[4], at::kFloat8_e4m3fn, dim, &p, &n_kv) || !want_scales(a[5], p.n_pages, n_kv) ||
      !want_scales(a[6], p.n_pages, n_kv) || !on_one_device(a, 7))
    return nullptr;
  p.head_dim = static_cast<uint32_t>(dim);
  p.n_kv_heads = n_kv;
  p.n_tokens = static_cast<uint32_t>(n);
  gdn_stream_t stream;
  if (!get_stream(args[7], a[0]->get_device(), &stream)) return nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(a[0]->get_device()));
  const int32_t *slots = static_cast<const int32_t *>(a[2].ptr());
  float *ks = static_cast<float *>(a[5].ptr()), *vs = static_cast<float *>(a[6].ptr());
  return finish(STORE ? gdn_kv_store_fp8(a[0].ptr(), a[1].ptr(), slots, a[3].ptr(), a[4].ptr(), ks, vs, &p, stream)
                      : gdn_kv_load_fp8(slots, a[3].ptr(), a[4].ptr(), ks, vs, a[0].ptr(), a[1].ptr(), &p, stream));
}

// Every entry: a C++ exception of torch (a tensor without storage, say) becomes a Python one.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *args, Py_ssize_t n) {
  try {
    return F(self, args, n);
  } catch (const std::exception &e) {
    if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return PyMethodDef{name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef g_methods[] = {method<py_kv_plan>("kv_plan"),
                           method<py_rope>("rope"),
                           method<py_rope_store>("rope_store"),
                           method<py_attn_workspace_size<false>>("attn_workspace_size"),
                           method<py_attn_paged<false>>("attn_paged"),
                           method<py_kv_fp8<true>>("kv_store_fp8"),
                           method<py_kv_fp8<false>>("kv_load_fp8"),
                           method<py_attn_workspace_size<true>>("attn_fp8_workspace_size"),
                           method<py_attn_paged<true>>("attn_paged_fp8"),
                           PyMethodDef{nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_paged_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged_binding() {
  PyObject *native = PyImport_ImportModule("serving_gdn_decode_gb300._native");
  if (!native) return nullptr;
  g_error = PyObject_GetAttrString(native, "GdnError");
  Py_DECREF(native);
  return g_error ? PyModule_Create(&g_module) : nullptr;
}
