"""Host-side tests of the 8-bit cache's C ABI and binding (no GPU needed): the
struct mirror, workspace sizes, and every argument check.

Calls pass made-up device addresses with exactly one thing wrong each, so they
are refused on the host; they are skipped where a CUDA device is visible.
"""
import ctypes

import pytest

from serving_gdn_decode_gb300 import _native as nat
from test_abi_host import no_device
from test_paged_host import L, addresses, attn_params, refused  # noqa: F401
import test_paged_host

KV = ("k", "v", "slot_map", "k_cache", "v_cache", "k_scale", "v_scale")
ATTN = ("q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "kv_lens", "token_start", "output")


def test_struct_mirror():
    test_paged_host.test_struct_mirrors("gdn_kv_fp8_params", nat.KvFp8Params)


def kv_params(**change):
    p = nat.KvFp8Params()
    for name, x in dict(dtype=1, head_dim=64, n_kv_heads=2, n_tokens=10, page_size=16, n_pages=20, k_stride=128, v_stride=128,
                        cache_page_stride=2048, cache_head_stride=1024, cache_slot_stride=64, **change).items():
        setattr(p, name, x)
    return p


def kv(L, store, params=None, **change):  # noqa: F811
    a = addresses(KV)
    a.update(change)
    p = kv_params()
    for name, x in (params or {}).items():
        setattr(p, name, x)
    order = KV if store else KV[2:] + KV[:2]
    return (L.gdn_kv_store_fp8 if store else L.gdn_kv_load_fp8)(*[a[n] for n in order], ctypes.byref(p), None)


@pytest.mark.parametrize("store", [True, False])
def test_kv_refusals(L, store):  # noqa: F811
    no_device()
    call = L.gdn_kv_store_fp8 if store else L.gdn_kv_load_fp8
    refused(call(*[1 << 30] * 7, None, None), "params is NULL")
    bad = nat.GDN_ERR_INVALID_ARGUMENT
    for name in KV:
        assert refused(kv(L, store, **{name: None}), name + " is NULL") == bad
        assert refused(kv(L, store, **{name: (5 << 34) + 1}), name + " must be") == bad
    for name in ("k_cache", "v_cache"):
        refused(kv(L, store, **{name: (5 << 34) + 8}), name + " must be 16-byte aligned")
    for params, text in ((dict(dtype=2), "dtype"), (dict(n_kv_heads=0), "> 0"), (dict(head_dim=0), "> 0"), (dict(n_pages=0), "> 0"),
                         (dict(page_size=0), "> 0"), (dict(n_kv_heads=16385), "heads"), (dict(n_tokens=(1 << 31) - (1 << 16) + 1), "n_tokens"),
                         (dict(n_pages=1 << 20, page_size=1 << 11), "2^31"), (dict(k_stride=127), "k_stride"), (dict(v_stride=127), "v_stride"),
                         (dict(k_stride=(1 << 40) + 1), "k_stride"), (dict(v_stride=-128), "v_stride"),
                         (dict(cache_slot_stride=63), "strides"), (dict(cache_page_stride=2056), "multiples of 16"),
                         (dict(cache_head_stride=1032), "multiples of 16"), (dict(cache_slot_stride=72), "multiples of 16"),
                         (dict(cache_page_stride=1 << 47), "strides")):
        assert refused(kv(L, store, params), text) == bad
    for dim in (8, 24, 272):
        assert refused(kv(L, store, dict(head_dim=dim, k_stride=1024, v_stride=1024, cache_slot_stride=512, cache_head_stride=8192,
                                         cache_page_stride=16384))) == nat.GDN_ERR_UNSUPPORTED
    a = addresses(KV)
    outs = KV[3:] if store else KV[:2]
    for o in outs:
        for i in KV:
            if i != o and {o, i} != {"k_cache", "v_cache"}:
                assert refused(kv(L, store, **{o: a[i]}), "overlaps") == bad
                assert refused(kv(L, store, **{o: a[i] + 16}), "overlaps") == bad
    assert kv(L, store, dict(n_tokens=0)) == nat.GDN_OK


def test_store_cache_rows(L):  # noqa: F811
    """Strides that let rows overlap; k_cache and v_cache among one another, as in gdn_rope_store."""
    no_device()
    refused(kv(L, True, dict(cache_slot_stride=1024, cache_head_stride=1024)), "overlap")
    refused(kv(L, True, dict(cache_page_stride=1024)), "overlap")
    a = addresses(KV)["k_cache"]
    apart = dict(cache_page_stride=4096)
    refused(kv(L, True, apart, v_cache=a), "overlaps")
    refused(kv(L, True, apart, v_cache=a + 1024), "overlaps")
    refused(kv(L, True, apart, v_cache=a + 2048 - 64), "overlaps")
    assert kv(L, True, dict(apart, n_tokens=0), v_cache=a + 2048) == nat.GDN_OK
    # what is only read may share rows; the outputs are refused after that check
    refused(kv(L, False, dict(cache_page_stride=1024), v_cache=a, k=None), "k is NULL")


def test_load_into_one_fused_row(L):  # noqa: F811
    """k and v as outputs may be views of one row per token, beside one another."""
    no_device()
    k = addresses(KV)["k"]
    fused = dict(k_stride=256, v_stride=256)
    refused(kv(L, False, fused, v=k + 2 * 127), "overlaps")
    refused(kv(L, False, fused, v=k + 2 * 128, slot_map=k + 2 * 128), "overlaps")


def attn(L, params=None, workspace=1 << 40, ws_bytes=1 << 30, **change):  # noqa: F811
    a = addresses(ATTN)
    a.update(change)
    p = attn_params()
    for name, x in (params or {}).items():
        setattr(p, name, x)
    return L.gdn_attn_paged_fp8(*[a[n] for n in ATTN], ctypes.byref(p), workspace, ws_bytes, None)


def size(L, **change):  # noqa: F811
    n = ctypes.c_size_t(0)
    p = attn_params(**change)
    return L.gdn_attn_fp8_workspace_size(ctypes.byref(p), ctypes.byref(n)), n.value


def test_attn_refusals(L):  # noqa: F811
    no_device()
    a = addresses(ATTN)
    bad = nat.GDN_ERR_INVALID_ARGUMENT
    for name in ATTN:
        if name != "token_start":
            assert refused(attn(L, **{name: None}), name + " is NULL") == bad
    for name in ATTN[1:3]:
        refused(attn(L, **{name: a[name] + 8}), name + " must be 16-byte aligned")
    for name in ATTN[:1] + ATTN[3:8]:
        refused(attn(L, **{name: a[name] + 2}), name + " must be 4-byte aligned")
    refused(attn(L, workspace=None), "workspace is NULL")
    refused(attn(L, workspace=(1 << 40) + 8), "workspace must be 16-byte aligned")
    status, need = size(L)
    assert status == nat.GDN_OK and need > 0
    refused(attn(L, ws_bytes=need - 1), "needed")
    for name in ATTN[:8]:
        assert refused(attn(L, output=a[name]), "overlaps") == bad
        assert refused(attn(L, workspace=a[name]), "overlaps") == bad
    refused(attn(L, workspace=a["output"]), "overlaps")
    for stride in ("cache_page_stride", "cache_head_stride", "cache_slot_stride"):
        good = getattr(attn_params(), stride)
        refused(attn(L, {stride: good + 8}), "multiples of 16")  # 16 bytes of a bf16 cache, 8 of this one
    for params, text in ((dict(dtype=2), "dtype"), (dict(n_q_heads=5), "multiple"), (dict(n_seqs=0), "> 0"), (dict(max_pages=0), "> 0"),
                         (dict(scale=float("nan")), "scale"), (dict(q_stride=8), "q_stride"), (dict(out_stride=8), "out_stride"),
                         (dict(max_pages=1 << 30), "max_pages")):
        assert refused(attn(L, params), text) == bad
    assert refused(attn(L, dict(head_dim=96))) == nat.GDN_ERR_UNSUPPORTED
    refused(L.gdn_attn_paged_fp8(*[1 << 30] * 9, None, 1 << 40, 1 << 30, None), "params is NULL")
    assert attn(L, dict(n_tokens=0)) == nat.GDN_OK


def test_attn_workspace_size(L):  # noqa: F811
    no_device()
    refused(L.gdn_attn_fp8_workspace_size(None, ctypes.byref(ctypes.c_size_t(0))), "NULL")
    refused(L.gdn_attn_fp8_workspace_size(ctypes.byref(attn_params()), None), "NULL")
    for change in (dict(n_pages=7), dict(page_size=24), dict(max_pages=900), dict(window=100), dict(cache_slot_stride=4096)):
        assert size(L, **change) == size(L)  # neither the cache nor the lengths matter


def tensors():
    import torch
    e = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    f8, i32 = torch.float8_e4m3fn, torch.int32
    return dict(k=e(5, 2, 64), v=e(5, 2, 64), slot_map=e(5, dtype=i32), k_cache=e(9, 2, 16, 64, dtype=f8), v_cache=e(9, 2, 16, 64, dtype=f8),
                k_scale=e(9, 2), v_scale=e(9, 2), q=e(5, 4, 64), block_table=e(5, 3, dtype=i32), kv_lens=e(5, dtype=i32),
                token_start=e(6, dtype=i32), output=e(5, 4, 64), workspace=e(100))


ORDER = {"store": KV, "load": KV[2:] + KV[:2], "attn": ATTN + ("workspace",)}


def call(op, **change):
    import serving_gdn_decode_gb300 as gdn
    t = {**tensors(), **change}
    f = {"store": gdn.gdn_kv_store_fp8, "load": gdn.gdn_kv_load_fp8, "attn": gdn.gdn_attn_paged_fp8}[op]
    return f(*[t[n] for n in ORDER[op]])


@pytest.mark.parametrize("op", ["store", "load", "attn"])
def test_binding_rules(L, op):  # noqa: F811
    """Everything but the device is right in `tensors`: CPU tensors are refused last, other faults before that."""
    import torch
    from serving_gdn_decode_gb300 import GdnError
    with pytest.raises(GdnError, match="CUDA tensor"):
        call(op)
    for name in ORDER[op]:
        with pytest.raises(TypeError, match=name):
            call(op, **{name: 3})
    t = tensors()
    faults = dict(k=[t["k"].to(torch.float16), t["k"][:, :1], t["k"][0], t["k"].transpose(0, 1), torch.zeros(5, 2, 128)[:, :, ::2]],
                  v=[t["v"].to(torch.bfloat16), t["v"][:4], t["v"].view(10, 64)],
                  slot_map=[t["slot_map"].long(), t["slot_map"][:4], t["slot_map"][None]],
                  k_cache=[t["k_cache"].view(torch.uint8), t["k_cache"].float(), t["k_cache"][:8], t["k_cache"][..., :32]],
                  v_cache=[t["v_cache"].view(torch.int8), t["v_cache"][:, :1], t["v_cache"][0]],
                  k_scale=[t["k_scale"].double(), t["k_scale"][:8], torch.zeros(9), torch.zeros(2, 9).t()],
                  v_scale=[t["v_scale"].to(torch.bfloat16), t["v_scale"][:, :1]],
                  q=[t["q"].to(torch.float16), t["q"][0], torch.zeros(5, 4, 96)], block_table=[t["block_table"].long(), t["block_table"][:4]],
                  kv_lens=[t["kv_lens"].long()], token_start=[t["token_start"][:5]], output=[t["output"].to(torch.bfloat16), t["output"][:4]])
    for name in ORDER[op]:
        for x in faults.get(name, []):
            with pytest.raises(GdnError) as e:
                call(op, **{name: x})
            assert "CUDA tensor" not in str(e.value)
    import serving_gdn_decode_gb300 as gdn
    q, k = t["q"], t["k_cache"]
    assert gdn.gdn_attn_fp8_workspace_size(q, k, 5) > 0
    with pytest.raises(GdnError):
        gdn.gdn_attn_fp8_workspace_size(q, k.float(), 5)
    with pytest.raises(GdnError):
        gdn.gdn_attn_workspace_size(q, k, 5)


def test_missing_binding_is_an_error_of_the_calls():
    import subprocess
    import sys
    code = ("import sys\nsys.modules['serving_gdn_decode_gb300._paged_binding'] = None\n"
            "from serving_gdn_decode_gb300 import gdn_kv_store_fp8, gdn_kv_load_fp8, gdn_attn_paged_fp8, gdn_attn_fp8_workspace_size\n"
            "for call in (lambda: gdn_kv_store_fp8(*[None] * 7), lambda: gdn_kv_load_fp8(*[None] * 7),\n"
            "             lambda: gdn_attn_paged_fp8(*[None] * 10), lambda: gdn_attn_fp8_workspace_size(None, None, 1)):\n"
            "    try:\n        call()\n    except RuntimeError as e:\n        assert 'missing' in str(e), e\n    else:\n        raise SystemExit('no error')\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
