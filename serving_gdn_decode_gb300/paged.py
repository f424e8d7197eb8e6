"""The full-attention layers of a hybrid model's serving step, on torch tensors:
``gdn_kv_plan``, ``gdn_rope``, ``gdn_rope_store``, ``gdn_attn_workspace_size``
and ``gdn_attn_paged`` of ``include/gdn.h``.

Argument marshalling only, as in ``_native``: shapes, strides and dtypes are
turned into the params struct of the C call, which checks the rest.  A call's
struct depends on nothing but shapes, strides, dtypes and scalars, so it is kept
for the next call with the same ones: a decode step is not paid for in Python.

The paged cache: ``k_cache`` and ``v_cache`` of shape [n_pages, n_kv_heads,
page_size, head_dim], f32 or bf16, with any strides over contiguous rows of
head_dim (pass ``cache.transpose(1, 2)`` for a cache held as [n_pages,
page_size, n_kv_heads, head_dim]).  Slot number: page * page_size + place in the page.

Every call runs on ``stream`` (default: the current stream of the tensors'
device) and does not block; tensors must stay alive and unchanged until the
stream reaches it.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._native import (GDN_ERR_INVALID_ARGUMENT, GDN_OK, AttnParams, GdnError, KvPlanParams,
                      RopeParams, gdn_last_error, lib)

DTYPE_F32, DTYPE_BF16 = 0, 1
ROPE_INTERLEAVED, ROPE_INVERSE = 0x1, 0x2
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}
_MAX_KEPT = 4096  # params structs kept, over all shapes

_kept: dict = {}


def _bad(message):
    return GdnError(GDN_ERR_INVALID_ARGUMENT, message)


def _looks(names, tensors):
    """What the params of a call depend on, for every tensor of it."""
    try:
        return tuple([(t.dtype, t.shape, t.stride(), t.get_device()) for t in tensors])
    except (AttributeError, TypeError):
        for name, t in zip(names, tensors):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor (got {type(t)})") from None
        raise


def _stream(stream, t):
    """The call's stream handle: `stream`, or the current one of t's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


_functions: dict = {}


def _function(name):
    """The library's function, looked up once."""
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(lib(), name)
    return f


def _keep(key, make):
    got = _kept.get(key)
    if got is None:
        made = make()
        if len(_kept) >= _MAX_KEPT:
            _kept.clear()
        got = _kept[key] = made
    return got


def _cuda(names, tensors):
    for name, t in zip(names, tensors):
        if not t.is_cuda:
            raise _bad(f"{name} must be a CUDA tensor")
        if t.device != tensors[0].device:
            raise _bad(f"{name} must be on {names[0]}'s device")


def _int32(name, t, shape):
    if t.dtype != torch.int32:
        raise _bad(f"{name} must be int32 (got {t.dtype})")
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise _bad(f"{name} must be contiguous of shape {tuple(shape)} (got {tuple(t.shape)})")


def _rows(name, t, dtype, shape):
    """[n_tokens, n_heads, head_dim] with contiguous rows; the token stride."""
    if t.dtype != dtype:
        raise _bad(f"{name} must be {dtype} (got {t.dtype})")
    if tuple(t.shape) != tuple(shape):
        raise _bad(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    heads, dim = shape[1], shape[2]
    if (dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != dim):
        raise _bad(f"{name}'s heads must be contiguous within a token")
    return t.stride(0) if shape[0] > 1 else heads * dim


def _cache(k_cache, v_cache, dtype, n_kv, dim):
    if k_cache.dim() != 4 or k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise _bad("k_cache and v_cache must be [n_pages, n_kv_heads, page_size, head_dim] of one layout")
    if k_cache.dtype != dtype or v_cache.dtype != dtype:
        raise _bad(f"k_cache and v_cache must be {dtype} (got {k_cache.dtype}, {v_cache.dtype})")
    n_pages, heads, page, d = k_cache.shape
    if d != dim or (n_kv is not None and heads != n_kv):
        raise _bad(f"k_cache has {heads} heads of {d}, expected {n_kv if n_kv is not None else heads} of {dim}")
    if d > 1 and k_cache.stride(3) != 1:
        raise _bad("the cache's rows of head_dim must be contiguous")
    # the stride of a dimension of size 1 says nothing
    strides = [s if n > 1 else d for s, n in zip(k_cache.stride()[:3], k_cache.shape[:3])]
    strides = [s if n > 1 else max(strides) for s, n in zip(strides, k_cache.shape[:3])]
    return n_pages, heads, page, (strides[0], strides[1], strides[2])


def _dtype(name, t):
    if t.dtype not in _DTYPES:
        raise _bad(f"{name} must be f32 or bf16 (got {t.dtype})")
    return _DTYPES[t.dtype]


def _failed(st):
    return GdnError(st, gdn_last_error())


# ------------------------------------------------------------------ plan

_PLAN = ("ctx_lens", "new_lens", "owned", "free_pages", "n_free", "block_table", "kv_lens", "owned_out",
         "n_free_out", "token_start", "slot_map", "positions")


def gdn_kv_plan(ctx_lens, new_lens, owned, free_pages, n_free, block_table, page_size, n_pages, kv_lens,
                owned_out, n_free_out, token_start, slot_map, positions, stream=None) -> None:
    """Bookkeeping of one step over a paged cache, on the device: takes pages for
    the requests' new tokens off the free stack into ``block_table`` ([n_seqs,
    max_pages], in place) and writes ``kv_lens``, ``owned_out``, ``n_free_out``,
    ``token_start`` (n_seqs + 1), and ``slot_map`` and ``positions`` of the packed
    new tokens (filled up with -1 and 0).  Contiguous int32 CUDA tensors; the
    outputs are arrays of their own (a loop swaps them with the inputs)."""
    tensors = (ctx_lens, new_lens, owned, free_pages, n_free, block_table, kv_lens, owned_out, n_free_out,
               token_start, slot_map, positions)

    def make():
        _cuda(_PLAN, tensors)
        n = ctx_lens.numel()
        if block_table.dim() != 2:
            raise _bad("block_table must be [n_seqs, max_pages]")
        shapes = ((n,), (n,), (n,), (free_pages.numel(),), (1,), (n, block_table.shape[1]), (n,), (n,), (1,),
                  (n + 1,), (slot_map.numel(),), (slot_map.numel(),))
        for name, t, shape in zip(_PLAN, tensors, shapes):
            _int32(name, t, shape)
        return ctypes.byref(KvPlanParams(n, page_size, n_pages, block_table.shape[1], free_pages.numel(),
                                         slot_map.numel()))

    p = _keep(("plan", page_size, n_pages, _looks(_PLAN, tensors)), make)
    st = _function("gdn_kv_plan")(*[t.data_ptr() for t in tensors], p, _stream(stream, ctx_lens))
    if st != GDN_OK:
        raise _failed(st)


# ------------------------------------------------------------------ rope

def _rope_params(q, k, v, positions, cos_sin, q_out, k_out, slot_map, k_cache, v_cache, axes, flags):
    store = v is not None
    dtype = _dtype("q", q)
    if q.dim() != 3 or k.dim() != 3:
        raise _bad("q and k must be [n_tokens, n_heads, head_dim]")
    n, n_q, dim = q.shape
    n_kv = k.shape[1]
    p = RopeParams()
    p.dtype, p.head_dim, p.n_q_heads, p.n_kv_heads, p.n_tokens, p.flags = dtype, dim, n_q, n_kv, n, flags
    p.q_stride = _rows("q", q, q.dtype, (n, n_q, dim))
    p.k_stride = _rows("k", k, q.dtype, (n, n_kv, dim))
    p.q_out_stride = _rows("q_out", q_out, q.dtype, (n, n_q, dim))
    if store:
        p.v_stride = _rows("v", v, q.dtype, (n, n_kv, dim))
        _int32("slot_map", slot_map, (n,))
        p.n_pages, _, p.page_size, (p.cache_page_stride, p.cache_head_stride, p.cache_slot_stride) = \
            _cache(k_cache, v_cache, q.dtype, n_kv, dim)
    else:
        p.k_out_stride = _rows("k_out", k_out, q.dtype, (n, n_kv, dim))
    if positions.dtype != torch.int32 or positions.dim() not in (1, 2) or positions.shape[-1] != n \
            or (n > 1 and positions.stride(-1) != 1):
        raise _bad("positions must be int32 [n_tokens] or [n_axes, n_tokens] with contiguous rows")
    p.n_axes = positions.shape[0] if positions.dim() == 2 else 1
    p.positions_stride = positions.stride(0) if positions.dim() == 2 and p.n_axes > 1 else 0
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise _bad("cos_sin must be contiguous f32 [n_positions, rot_dim]")
    p.n_positions, p.rot_dim = cos_sin.shape
    if axes is not None:
        if len(axes) != p.rot_dim // 2:
            raise _bad(f"axes has {len(axes)} entries, expected rot_dim / 2 = {p.rot_dim // 2}")
        if p.rot_dim <= 2 * len(p.axis_of_pair):
            for j, a in enumerate(axes):
                p.axis_of_pair[j] = a
    return p


_ROPE = ("q", "k", "positions", "cos_sin", "q_out", "k_out")
_STORE = ("q", "k", "v", "positions", "cos_sin", "slot_map", "q_out", "k_cache", "v_cache")


def gdn_rope(q, k, positions, cos_sin, q_out, k_out, axes=None, interleaved=False, inverse=False,
             stream=None) -> None:
    """Rotary positions on q [n_tokens, n_q_heads, head_dim] and k [n_tokens,
    n_kv_heads, head_dim] (views of a fused projection are fine), into ``q_out``
    and ``k_out`` (may be q and k).  ``positions``: int32 [n_axes, n_tokens], or
    [n_tokens] for one axis; ``axes``: the axis of each of the rot_dim / 2 pairs
    (``bytes``; default: all axis 0); ``cos_sin``: f32 [n_positions, rot_dim],
    cosines then sines.  ``inverse`` applies the inverse rotation: the gradients
    of q and k from those of q_out and k_out."""
    tensors = (q, k, positions, cos_sin, q_out, k_out)
    flags = (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0)
    if axes is not None and type(axes) is not bytes:
        axes = bytes(axes)

    def make():
        _cuda(_ROPE, tensors)
        return ctypes.byref(_rope_params(q, k, None, positions, cos_sin, q_out, k_out, None, None, None, axes, flags))

    p = _keep(("rope", flags, axes, _looks(_ROPE, tensors)), make)
    st = _function("gdn_rope")(*[t.data_ptr() for t in tensors], p, _stream(stream, q))
    if st != GDN_OK:
        raise _failed(st)


def gdn_rope_store(q, k, v, positions, cos_sin, slot_map, k_cache, v_cache, q_out, axes=None,
                   interleaved=False, stream=None) -> None:
    """``gdn_rope`` whose k goes, with v beside it, into the paged cache at
    ``slot_map`` (int32 [n_tokens]; -1: nowhere)."""
    tensors = (q, k, v, positions, cos_sin, slot_map, q_out, k_cache, v_cache)
    flags = ROPE_INTERLEAVED if interleaved else 0
    if axes is not None and type(axes) is not bytes:
        axes = bytes(axes)

    def make():
        _cuda(_STORE, tensors)
        return ctypes.byref(_rope_params(q, k, v, positions, cos_sin, q_out, None, slot_map, k_cache, v_cache, axes,
                                         flags))

    p = _keep(("store", flags, axes, _looks(_STORE, tensors)), make)
    st = _function("gdn_rope_store")(*[t.data_ptr() for t in tensors], p, _stream(stream, q))
    if st != GDN_OK:
        raise _failed(st)


# ------------------------------------------------------------------ attention

def _attn_params(q, k_cache, v_cache, n_seqs, max_pages, out_stride, scale, window):
    dtype = _dtype("q", q)
    if q.dim() != 3:
        raise _bad("q must be [n_tokens, n_q_heads, head_dim]")
    n, n_q, dim = q.shape
    p = AttnParams()
    p.dtype, p.head_dim, p.n_q_heads, p.n_tokens, p.n_seqs, p.max_pages = dtype, dim, n_q, n, n_seqs, max_pages
    p.n_pages, p.n_kv_heads, p.page_size, (p.cache_page_stride, p.cache_head_stride, p.cache_slot_stride) = \
        _cache(k_cache, v_cache, q.dtype, None, dim)
    p.window = window
    p.scale = 1.0 / math.sqrt(dim) if scale is None else scale
    p.q_stride = _rows("q", q, q.dtype, q.shape)
    p.out_stride = n_q * dim if out_stride is None else out_stride
    return p


def gdn_attn_workspace_size(q, k_cache, n_seqs) -> int:
    """Bytes of workspace ``gdn_attn_paged`` needs for ``n_seqs`` requests with
    q's rows and heads; the lengths do not matter."""
    p = _attn_params(q, k_cache, k_cache, n_seqs, 1, None, None, 0)
    out = ctypes.c_size_t()
    st = lib().gdn_attn_workspace_size(ctypes.byref(p), ctypes.byref(out))
    if st != GDN_OK:
        raise _failed(st)
    return out.value


_ATTN = ("q", "k_cache", "v_cache", "block_table", "kv_lens", "token_start", "output", "workspace")


def gdn_attn_paged(q, k_cache, v_cache, block_table, kv_lens, token_start, output, workspace, scale=None,
                   window=0, stream=None) -> None:
    """Attention of each request's newest tokens over its paged cache.  q and
    output: [n_tokens, n_q_heads, head_dim]; ``block_table`` int32 [n_seqs,
    max_pages], ``kv_lens`` int32 [n_seqs] (the step's tokens among them),
    ``token_start`` int32 [n_seqs + 1] (None: one token per request).  ``scale``
    defaults to 1/sqrt(head_dim); ``window`` > 0 limits a token to its last
    keys.  ``workspace``: a contiguous CUDA tensor of at least
    ``gdn_attn_workspace_size`` bytes."""
    ragged = token_start is not None
    tensors = (q, k_cache, v_cache, block_table, kv_lens, token_start if ragged else kv_lens, output, workspace)

    def make():
        _cuda(_ATTN, tensors)
        n = kv_lens.numel()
        if block_table.dim() != 2:
            raise _bad("block_table must be [n_seqs, max_pages]")
        _int32("block_table", block_table, (n, block_table.shape[1]))
        _int32("kv_lens", kv_lens, (n,))
        if ragged:
            _int32("token_start", token_start, (n + 1,))
        if not workspace.is_contiguous():
            raise _bad("workspace must be a contiguous CUDA tensor")
        _dtype("q", q)
        if q.dim() != 3:
            raise _bad("q must be [n_tokens, n_q_heads, head_dim]")
        out_stride = _rows("output", output, q.dtype, q.shape)
        return (ctypes.byref(_attn_params(q, k_cache, v_cache, n, block_table.shape[1], out_stride, scale, window)),
                workspace.numel() * workspace.element_size())

    p, ws_bytes = _keep(("attn", ragged, scale, window, _looks(_ATTN, tensors)), make)
    st = _function("gdn_attn_paged")(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
                                     kv_lens.data_ptr(), token_start.data_ptr() if ragged else None,
                                     output.data_ptr(), p, workspace.data_ptr(), ws_bytes, _stream(stream, q))
    if st != GDN_OK:
        raise _failed(st)
