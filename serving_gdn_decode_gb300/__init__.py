"""GB300-native (sm_103a) Gated DeltaNet recurrence: decode, per-token state
capture for speculative-decode rollback, and long prefill; and the part of a
hybrid model's full-attention layers that a serving step needs: the plan of a
paged key-value cache, rotary positions with the store, and paged attention,
over caches of f32, bf16 or 8-bit codes with block scales.

The compute lives in ``libgdn_gb300.so`` (CUDA kernels behind the C ABI of
``include/gdn.h``); this package is its thin Python binding plus the
parameter packer and the seeded synthetic-input generator.
"""
from .params import (FLAG_DECAY_AFTER, FLAG_KHEAD_DIV, N_PARAMS, PATH_AUTO, PATH_CHUNKED,
                     PATH_CHUNKED_TF32, PATH_SCAN, pack_params, q_scale_bits)

__all__ = ["FLAG_DECAY_AFTER", "FLAG_KHEAD_DIV", "N_PARAMS", "PATH_AUTO", "PATH_CHUNKED",
           "PATH_CHUNKED_TF32", "PATH_SCAN", "pack_params", "q_scale_bits", "gdn_forward", "gdn_forward_capture",
           "gdn_last_error", "gdn_path_name", "gdn_commit_capture", "gdn_forward_layers",
           "gdn_forward_host", "gdn_forward_ws", "gdn_workspace_size", "HostPipeline", "GdnError",
           "gdn_kv_plan", "gdn_rope", "gdn_rope_store", "gdn_attn_workspace_size", "gdn_attn_paged",
           "gdn_kv_store_fp8", "gdn_kv_load_fp8", "gdn_attn_fp8_workspace_size", "gdn_attn_paged_fp8"]

_NATIVE = ("gdn_forward", "gdn_forward_capture", "gdn_last_error", "gdn_path_name",
           "gdn_commit_capture", "gdn_forward_layers", "gdn_forward_host", "gdn_forward_ws",
           "gdn_workspace_size", "HostPipeline", "GdnError")
_PAGED = ("gdn_kv_plan", "gdn_rope", "gdn_rope_store", "gdn_attn_workspace_size", "gdn_attn_paged",
          "gdn_kv_store_fp8", "gdn_kv_load_fp8", "gdn_attn_fp8_workspace_size", "gdn_attn_paged_fp8")


def __getattr__(name):
    # The native binding loads on first use, so importing the package (for
    # the parameter packer or the input generator) needs no GPU library.
    if name in _NATIVE:
        from . import _native
        return getattr(_native, name)
    if name in _PAGED:
        from . import paged
        globals()[name] = getattr(paged, name)  # found without this function from now on
        return globals()[name]
    raise AttributeError(name)
