"""The full-attention layers of a hybrid model's serving step, on torch tensors:
``gdn_kv_plan``, ``gdn_rope``, ``gdn_rope_store``, ``gdn_attn_workspace_size``
and ``gdn_attn_paged`` of ``include/gdn.h``, and with an 8-bit cache
``gdn_kv_store_fp8``, ``gdn_kv_load_fp8``, ``gdn_attn_fp8_workspace_size`` and
``gdn_attn_paged_fp8``.

Argument marshalling only, as in ``_native``, here by the compiled module
``_paged_binding``: shapes, strides and dtypes become the params struct of the C
call, which checks the rest.  There is no fallback: if the module is missing or
cannot load, every call raises.

The paged cache: ``k_cache`` and ``v_cache`` of shape [n_pages, n_kv_heads,
page_size, head_dim], f32 or bf16, with any strides over contiguous rows of
head_dim (pass ``cache.transpose(1, 2)`` for a cache held as [n_pages,
page_size, n_kv_heads, head_dim]).  Slot number: page * page_size + place in the page.
An 8-bit cache has ``k_cache`` and ``v_cache`` of ``torch.float8_e4m3fn`` and, for
each page and key head, an f32 scale in ``k_scale`` and ``v_scale`` ([n_pages,
n_kv_heads], contiguous): an element stands for code * scale.

Every call runs on ``stream`` (default: the current stream of the tensors'
device) and does not block; tensors must stay alive and unchanged until the
stream reaches it.  No call is recorded by autograd, and a tensor written in place
keeps its version: the gradients of ``gdn_rope`` are a call of their own.
"""
from __future__ import annotations

try:
    from . import _paged_binding as _binding
except ImportError as e:
    class _Missing:
        def __init__(self, cause):
            self._cause = cause

        def __getattr__(self, name):
            raise RuntimeError("_paged_binding.so is missing or cannot load: build it with "
                               "`python -m serving_gdn_decode_gb300.build` (there is no fallback)") from self._cause

    _binding = _Missing(e)

DTYPE_F32, DTYPE_BF16 = 0, 1
ROPE_INTERLEAVED, ROPE_INVERSE = 0x1, 0x2


def gdn_kv_plan(ctx_lens, new_lens, owned, free_pages, n_free, block_table, page_size, n_pages, kv_lens,
                owned_out, n_free_out, token_start, slot_map, positions, stream=None) -> None:
    """Bookkeeping of one step over a paged cache, on the device: takes pages for
    the requests' new tokens off the free stack into ``block_table`` ([n_seqs,
    max_pages], in place) and writes ``kv_lens``, ``owned_out``, ``n_free_out``,
    ``token_start`` (n_seqs + 1), and ``slot_map`` and ``positions`` of the packed
    new tokens (filled up with -1 and 0).  Contiguous int32 CUDA tensors; the
    outputs are arrays of their own (a loop swaps them with the inputs)."""
    _binding.kv_plan(ctx_lens, new_lens, owned, free_pages, n_free, block_table, kv_lens, owned_out, n_free_out,
                     token_start, slot_map, positions, page_size, n_pages, stream)


def _axes(axes):
    return axes if axes is None or type(axes) is bytes else bytes(axes)


def gdn_rope(q, k, positions, cos_sin, q_out, k_out, axes=None, interleaved=False, inverse=False,
             stream=None) -> None:
    """Rotary positions on q [n_tokens, n_q_heads, head_dim] and k [n_tokens,
    n_kv_heads, head_dim] (views of a fused projection are fine), into ``q_out``
    and ``k_out`` (may be q and k).  ``positions``: int32 [n_axes, n_tokens], or
    [n_tokens] for one axis; ``axes``: the axis of each of the rot_dim / 2 pairs
    (``bytes``; default: all axis 0); ``cos_sin``: f32 [n_positions, rot_dim],
    cosines then sines.  ``inverse`` applies the inverse rotation: the gradients
    of q and k from those of q_out and k_out."""
    _binding.rope(q, k, positions, cos_sin, q_out, k_out, _axes(axes),
                  (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0), stream)


def gdn_rope_store(q, k, v, positions, cos_sin, slot_map, k_cache, v_cache, q_out, axes=None,
                   interleaved=False, stream=None) -> None:
    """``gdn_rope`` whose k goes, with v beside it, into the paged cache at
    ``slot_map`` (int32 [n_tokens]; -1: nowhere)."""
    _binding.rope_store(q, k, v, positions, cos_sin, slot_map, q_out, k_cache, v_cache, _axes(axes),
                        ROPE_INTERLEAVED if interleaved else 0, stream)


def gdn_attn_workspace_size(q, k_cache, n_seqs) -> int:
    """Bytes of workspace ``gdn_attn_paged`` needs for ``n_seqs`` requests with
    q's rows and heads; the lengths do not matter."""
    return _binding.attn_workspace_size(q, k_cache, n_seqs)


def gdn_attn_paged(q, k_cache, v_cache, block_table, kv_lens, token_start, output, workspace, scale=None,
                   window=0, stream=None) -> None:
    """Attention of each request's newest tokens over its paged cache.  q and
    output: [n_tokens, n_q_heads, head_dim]; ``block_table`` int32 [n_seqs,
    max_pages], ``kv_lens`` int32 [n_seqs] (the step's tokens among them),
    ``token_start`` int32 [n_seqs + 1] (None: one token per request).  ``scale``
    defaults to 1/sqrt(head_dim); ``window`` > 0 limits a token to its last
    keys.  ``workspace``: a contiguous CUDA tensor of at least
    ``gdn_attn_workspace_size`` bytes."""
    _binding.attn_paged(q, k_cache, v_cache, block_table, kv_lens, token_start, output, workspace, scale, window,
                        stream)


def gdn_kv_store_fp8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream=None) -> None:
    """Quantises k and v ([n_tokens, n_kv_heads, head_dim], f32 or bf16) as they are
    written to the 8-bit paged cache at ``slot_map`` (int32 [n_tokens], as
    ``gdn_kv_plan`` gives it; negative: nowhere).  A page's scale per key head is the
    smallest power of two that keeps its tokens within e4m3's range; it starts anew
    with the page's first token and grows with later ones, the codes before them
    rounded again.  Tokens of one page must be neighbours, slot after slot."""
    _binding.kv_store_fp8(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, stream)


def gdn_kv_load_fp8(slot_map, k_cache, v_cache, k_scale, v_scale, k, v, stream=None) -> None:
    """Rows of the 8-bit cache as values: row i of ``k`` and ``v`` ([n_tokens,
    n_kv_heads, head_dim], f32 or bf16) from slot ``slot_map[i]``; rows of negative
    slots are left as they were."""
    _binding.kv_load_fp8(slot_map, k_cache, v_cache, k_scale, v_scale, k, v, stream)


def gdn_attn_fp8_workspace_size(q, k_cache, n_seqs) -> int:
    """Bytes of workspace ``gdn_attn_paged_fp8`` needs for ``n_seqs`` requests with
    q's rows and heads; the lengths do not matter."""
    return _binding.attn_fp8_workspace_size(q, k_cache, n_seqs)


def gdn_attn_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, token_start, output,
                       workspace, scale=None, window=0, stream=None) -> None:
    """``gdn_attn_paged`` over an 8-bit cache; q and output are f32 or bf16, and
    ``workspace`` has at least ``gdn_attn_fp8_workspace_size`` bytes."""
    _binding.attn_paged_fp8(q, k_cache, v_cache, k_scale, v_scale, block_table, kv_lens, token_start, output,
                            workspace, scale, window, stream)
