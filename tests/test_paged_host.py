"""Host-side tests of the full-attention operators' C ABI and binding (no GPU
needed): struct mirrors, workspace sizes, and every argument check.

Calls pass made-up device addresses with exactly one thing wrong each, so they
are refused on the host; they are skipped where a CUDA device is visible.
"""
import ctypes
import re

import numpy as np
import pytest

from serving_gdn_decode_gb300 import _native as nat
from test_abi_host import no_device


@pytest.fixture(scope="module")
def L():
    from serving_gdn_decode_gb300 import build
    build.build()
    return nat.lib()


def header():
    text = open(nat.HEADER_PATH).read()
    return re.sub(r"/\*.*?\*/", "", text, flags=re.S), text


@pytest.mark.parametrize("name,cls", [("gdn_kv_plan_params", nat.KvPlanParams), ("gdn_rope_params", nat.RopeParams),
                                      ("gdn_attn_params", nat.AttnParams)])
def test_struct_mirrors(name, cls):
    body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), header()[0], re.S).group(1)
    kinds = {"uint32_t": ctypes.c_uint32, "int64_t": ctypes.c_int64, "float": ctypes.c_float, "uint8_t": ctypes.c_uint8}
    want = []
    for kind, names in re.findall(r"(uint32_t|int64_t|float|uint8_t)\s+([^;]+);", body):
        for n in names.split(","):
            n = n.strip()
            want.append((n.split("[")[0], kinds[kind] * 128 if "[" in n else kinds[kind]))
    assert [n for n, _ in cls._fields_] == [n for n, _ in want]
    for (_, a), (_, b) in zip(cls._fields_, want):
        assert ctypes.sizeof(a) == ctypes.sizeof(b)


def test_constants():
    text = header()[1]
    for name, val in (("OUT_OF_PAGES", 0x2), ("BAD_REQUEST", 0x4), ("BAD_PAGE", 0x8), ("BAD_POSITION", 0x10)):
        assert re.search(r"#define GDN_DEVICE_%s 0x%xu" % (name, val), text)
        assert getattr(nat, "GDN_DEVICE_" + name) == val
    for line in ("GDN_DTYPE_F32 0u", "GDN_DTYPE_BF16 1u", "GDN_ROPE_INTERLEAVED 0x1u", "GDN_ROPE_INVERSE 0x2u",
                 "GDN_ROPE_MAX_DIM 256u"):
        assert "#define " + line in text
    from serving_gdn_decode_gb300 import paged
    assert (paged.DTYPE_F32, paged.DTYPE_BF16, paged.ROPE_INTERLEAVED, paged.ROPE_INVERSE) == (0, 1, 1, 2)


# ------------------------------------------------------------------ calls with made-up addresses


def refused(status, text=""):
    assert status in (nat.GDN_ERR_INVALID_ARGUMENT, nat.GDN_ERR_UNSUPPORTED), status
    assert text in nat.gdn_last_error(), nat.gdn_last_error()
    return status


def addresses(names, step=1 << 30):
    return {n: (i + 1) * step for i, n in enumerate(names)}


PLAN = ("ctx_lens", "new_lens", "owned", "free_pages", "n_free", "block_table", "kv_lens", "owned_out", "n_free_out",
        "token_start", "slot_map", "positions")


def plan(L, params=None, **change):
    a = addresses(PLAN)
    a.update(change)
    p = nat.KvPlanParams(8, 16, 100, 10, 50, 40)
    for k, v in (params or {}).items():
        setattr(p, k, v)
    return L.gdn_kv_plan(*[a[n] for n in PLAN], ctypes.byref(p), None)


@no_device
def test_plan_refusals(L):
    for n in PLAN:
        assert refused(plan(L, **{n: None}), n) == nat.GDN_ERR_INVALID_ARGUMENT
        refused(plan(L, **{n: (1 << 40) + 2}), "4-byte aligned")
    for n in ("n_seqs", "page_size", "n_pages", "max_pages"):
        refused(plan(L, {n: 0}), "> 0")
    refused(plan(L, {"n_pages": 1 << 27}), "2^31")
    refused(plan(L, {"max_pages": 1 << 28}), "2^31")
    refused(plan(L, {"n_slots": (1 << 31) - 5}), "2^31")
    a = addresses(PLAN)
    refused(plan(L, kv_lens=a["ctx_lens"]), "kv_lens overlaps ctx_lens")
    refused(plan(L, owned_out=a["owned"] + 4), "owned_out overlaps owned")
    refused(plan(L, n_free_out=a["n_free"]), "n_free_out overlaps n_free")
    refused(plan(L, slot_map=a["positions"] + 156), "overlaps")
    refused(plan(L, token_start=a["kv_lens"] - 32), "overlaps")  # n_seqs + 1 entries
    assert L.gdn_kv_plan(*[a[n] for n in PLAN], None, None) == nat.GDN_ERR_INVALID_ARGUMENT


def rope_params(store=True, **change):
    p = nat.RopeParams()
    base = dict(dtype=1, head_dim=64, rot_dim=32, n_q_heads=4, n_kv_heads=2, n_tokens=10, n_axes=2, n_positions=100,
                flags=0, page_size=8 if store else 0, n_pages=20 if store else 0, q_stride=256, k_stride=128,
                v_stride=128, q_out_stride=256, k_out_stride=128, positions_stride=10, cache_page_stride=1024,
                cache_head_stride=512, cache_slot_stride=64)
    base.update(change)
    axes = base.pop("axes", [0, 1] * 8)
    for k, v in base.items():
        setattr(p, k, v)
    for j, a in enumerate(axes):
        p.axis_of_pair[j] = a
    return p


ROPE = ("q", "k", "positions", "cos_sin", "q_out", "k_out")
STORE = ("q", "k", "v", "positions", "cos_sin", "slot_map", "q_out", "k_cache", "v_cache")


def rope(L, store, params=None, **change):
    names = STORE if store else ROPE
    a = addresses(names)
    a.update(change)
    p = rope_params(store, **(params or {}))
    return (L.gdn_rope_store if store else L.gdn_rope)(*[a[n] for n in names], ctypes.byref(p), None)


@no_device
@pytest.mark.parametrize("store", [False, True])
def test_rope_refusals(L, store):
    names = STORE if store else ROPE
    for n in names:
        refused(rope(L, store, **{n: None}), n + " is NULL")
        refused(rope(L, store, **{n: (1 << 40) + 1}), "aligned")
    for change, text in (({"dtype": 2}, "dtype"), ({"flags": 4}, "flag bits"), ({"head_dim": 0}, "head_dim"),
                         ({"head_dim": 258}, "head_dim"), ({"head_dim": 63}, "head_dim"), ({"rot_dim": 0}, "rot_dim"),
                         ({"rot_dim": 66}, "rot_dim"), ({"rot_dim": 15}, "rot_dim"), ({"n_q_heads": 0}, "> 0"),
                         ({"n_kv_heads": 0}, "> 0"), ({"n_axes": 0}, "> 0"), ({"n_positions": 0}, "> 0"),
                         ({"n_axes": 1}, "axis_of_pair[1]"), ({"q_stride": 255}, "q_stride"),
                         ({"k_stride": 127}, "k_stride"), ({"q_out_stride": -256}, "q_out_stride"),
                         ({"v_stride" if store else "k_out_stride": 1}, "stride"), ({"positions_stride": -1}, "positions_stride"),
                         ({"n_tokens": 1 << 31}, "2^31")):
        refused(rope(L, store, change), text)
    a = addresses(names)
    refused(rope(L, store, q_out=a["q"] + 2), "q_out overlaps q")
    refused(rope(L, store, q_out=a["k"] + 100), "q_out overlaps k")
    refused(rope(L, store, {"q_out_stride": 300}, q_out=a["q"]), "q_out overlaps q")  # in place needs one layout
    refused(rope(L, store, q_out=a["cos_sin"] + 12800 - 4), "q_out overlaps cos_sin")
    if store:
        assert refused(rope(L, True, {"flags": 2})) == nat.GDN_ERR_UNSUPPORTED
        for change, text in (({"page_size": 0}, "> 0"), ({"n_pages": 0}, "> 0"), ({"n_pages": 1 << 29}, "2^31"),
                             ({"cache_slot_stride": 63}, "strides"), ({"cache_page_stride": 1 << 47}, "strides")):
            refused(rope(L, True, change), text)
        refused(rope(L, True, k_cache=a["v"]), "k_cache overlaps v")
        refused(rope(L, True, v_cache=a["k_cache"]), "v_cache overlaps k_cache")
        refused(rope(L, True, v_cache=a["slot_map"] + 36), "v_cache overlaps slot_map")
    else:
        refused(rope(L, False, k_out=a["q"]), "k_out overlaps q")
        refused(rope(L, False, k_out=a["q_out"] + 512), "k_out overlaps q_out")
    # no tokens: nothing to check on the buffers, nothing to do
    assert rope(L, store, {"n_tokens": 0}, **{n: None for n in names}) == nat.GDN_OK


@no_device
def test_rope_fused_rows_do_not_overlap(L):
    """In place in the rows of a fused projection: q_out lies among k's and v's bytes without touching them.
    Moved by an element, it does touch k."""
    row, base = 512, 1 << 40
    wide = {"q_stride": row, "k_stride": row, "v_stride": row, "q_out_stride": row}
    ok = dict(q=base, q_out=base, k=base + 2 * 256, v=base + 2 * 384)
    # refused for another reason only: the aligned check on positions comes after no overlap was found... so ask for it
    refused(rope(L, True, wide, **{**ok, "q_out": base + 4}), "q_out overlaps q")
    refused(rope(L, True, wide, **{**ok, "q": base + (1 << 39), "q_out": base + 4}), "q_out overlaps k")
    refused(rope(L, True, wide, **{**ok, "v_cache": base + 2 * 448}), "v_cache overlaps")


ATTN = ("q", "k_cache", "v_cache", "block_table", "kv_lens", "token_start", "output")


def attn_params(**change):
    p = nat.AttnParams()
    base = dict(dtype=1, head_dim=128, n_q_heads=8, n_kv_heads=2, n_seqs=4, n_tokens=6, page_size=16, n_pages=50,
                max_pages=9, window=0, scale=0.1, q_stride=1024, out_stride=1024, cache_page_stride=4096,
                cache_head_stride=2048, cache_slot_stride=128)
    base.update(change)
    for k, v in base.items():
        setattr(p, k, v)
    return p


def attn(L, params=None, workspace=1 << 40, ws_bytes=1 << 30, **change):
    a = addresses(ATTN)
    a.update(change)
    p = attn_params(**(params or {}))
    return L.gdn_attn_paged(*[a[n] for n in ATTN], ctypes.byref(p), workspace, ws_bytes, None)


def workspace_size(L, **change):
    out = ctypes.c_size_t()
    p = attn_params(**change)
    st = L.gdn_attn_workspace_size(ctypes.byref(p), ctypes.byref(out))
    return st, out.value


@no_device
def test_attn_refusals(L):
    for n in ATTN:
        if n != "token_start":
            refused(attn(L, **{n: None}), n + " is NULL")
        refused(attn(L, **{n: (1 << 41) + 1}), "aligned")
    refused(attn(L, q=(1 << 41) + 2), "q must be 4-byte aligned")
    refused(attn(L, k_cache=(1 << 41) + 8), "k_cache must be 16-byte aligned")
    for change, text in (({"dtype": 7}, "dtype"), ({"n_q_heads": 0}, "> 0"), ({"n_kv_heads": 0}, "> 0"), ({"n_seqs": 0}, "> 0"),
                         ({"max_pages": 0}, "> 0"), ({"head_dim": 0}, "> 0"), ({"n_pages": 0}, "> 0"), ({"page_size": 0}, "> 0"),
                         ({"n_kv_heads": 3}, "multiple"), ({"scale": float("nan")}, "scale"), ({"scale": float("inf")}, "scale"),
                         ({"cache_slot_stride": 132}, "16 bytes"), ({"cache_head_stride": 2052}, "16 bytes"),
                         ({"cache_page_stride": 4100}, "16 bytes"), ({"q_stride": 1023}, "q_stride"),
                         ({"out_stride": 8}, "out_stride"), ({"q_stride": 1025}, "even"), ({"n_pages": 1 << 28}, "2^31"),
                         ({"max_pages": 1 << 28}, "2^31"), ({"n_tokens": 1 << 28}, "2^31")):
        assert refused(attn(L, change), text) == nat.GDN_ERR_INVALID_ARGUMENT
        assert workspace_size(L, **change)[0] == nat.GDN_ERR_INVALID_ARGUMENT
    for dim in (32, 96, 512, 127):
        assert refused(attn(L, {"head_dim": dim, "q_stride": 8 * dim, "out_stride": 8 * dim, "cache_slot_stride": 512}),
                       "head_dim") == nat.GDN_ERR_UNSUPPORTED
    refused(attn(L, {"n_tokens": 3}, token_start=None), "token_start")
    a = addresses(ATTN)
    refused(attn(L, output=a["q"]), "output overlaps q")
    refused(attn(L, output=a["k_cache"] + 4096), "output overlaps k_cache")
    refused(attn(L, workspace=None), "workspace is NULL")
    refused(attn(L, ws_bytes=1000), "workspace has 1000 bytes")
    refused(attn(L, workspace=(1 << 40) + 8), "workspace must be 16-byte aligned")
    refused(attn(L, workspace=a["v_cache"]), "workspace overlaps v_cache")
    refused(attn(L, workspace=a["output"]), "workspace overlaps output")
    # no rows: nothing to do
    assert attn(L, {"n_tokens": 0}) == nat.GDN_OK


def test_attn_workspace_size(L):
    """A function of types and sizes alone; it grows with the rows of a tile, and stays in megabytes."""
    st, base = workspace_size(L)
    assert st == nat.GDN_OK and 0 < base < 64 << 20 and base % 16 == 0
    assert workspace_size(L, n_pages=1000, max_pages=400, page_size=64)[1] == base
    assert workspace_size(L, n_tokens=4 * 16)[1] > base
    for dtype in (0, 1):
        for dim in (64, 128, 256):
            st, n = workspace_size(L, dtype=dtype, head_dim=dim, q_stride=8 * dim, out_stride=8 * dim, cache_slot_stride=dim,
                                   cache_head_stride=16 * dim, cache_page_stride=32 * dim, n_tokens=64)
            assert st == nat.GDN_OK and 0 < n < 64 << 20
    assert L.gdn_attn_workspace_size(ctypes.byref(attn_params()), None) == nat.GDN_ERR_INVALID_ARGUMENT


# ------------------------------------------------------------------ the torch binding


def shapes(op):
    """Arguments of a call that is right but for being on the host: refused as such, after every other check."""
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    if op == "kv_plan":
        return dict(ctx_lens=i(2), new_lens=i(2), owned=i(2), free_pages=i(4), n_free=i(1), block_table=i(2, 3),
                    page_size=8, n_pages=5, kv_lens=i(2), owned_out=i(2), n_free_out=i(1), token_start=i(3),
                    slot_map=i(7), positions=i(7))
    f = torch.zeros
    if op == "rope":
        return dict(q=f(2, 4, 64), k=f(2, 1, 64), positions=i(3, 2), cos_sin=f(9, 32), q_out=f(2, 4, 64),
                    k_out=f(2, 1, 64), axes=[0, 2] * 8)
    if op == "rope_store":
        return dict(q=f(2, 4, 64), k=f(2, 2, 64), v=f(2, 2, 64), positions=i(2), cos_sin=f(9, 64), slot_map=i(2),
                    k_cache=f(5, 2, 8, 64), v_cache=f(5, 2, 8, 64), q_out=f(2, 4, 64))
    return dict(q=f(2, 4, 64), k_cache=f(5, 2, 8, 64), v_cache=f(5, 2, 8, 64), block_table=i(2, 3), kv_lens=i(2),
                token_start=i(3), output=f(2, 4, 64), workspace=f(10))


def call(op, **change):
    import serving_gdn_decode_gb300 as gdn
    a = shapes(op)
    a.update(change)
    return getattr(gdn, "gdn_" + op)(**a)


@pytest.mark.parametrize("op", ["kv_plan", "rope", "rope_store", "attn_paged"])
def test_binding_takes_cuda_tensors_only(L, op):
    import torch
    with pytest.raises(nat.GdnError, match="must be a CUDA tensor") as e:
        call(op)
    assert e.value.status == nat.GDN_ERR_INVALID_ARGUMENT
    for name, x in shapes(op).items():
        if isinstance(x, torch.Tensor):
            with pytest.raises(TypeError, match=name):
                call(op, **{name: [1, 2]})
            with pytest.raises(nat.GdnError, match=name):
                call(op, **{name: x.to(torch.float64) if name != "workspace" else torch.zeros(4, 4).t()[::2]})


def test_binding_shape_rules(L):
    import torch
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    f = torch.zeros

    def refuse(op, text, **change):
        with pytest.raises(nat.GdnError, match=text):
            call(op, **change)

    refuse("kv_plan", "new_lens", new_lens=i(3))
    refuse("kv_plan", "block_table", block_table=i(6))
    refuse("kv_plan", "block_table", block_table=i(3, 2).t())
    refuse("kv_plan", "token_start", token_start=i(2))
    refuse("kv_plan", "positions", positions=i(6))
    refuse("kv_plan", "n_free", n_free=i(2))
    refuse("kv_plan", "page_size", page_size=-1)
    refuse("rope", "k must", k=f(3, 1, 64))
    refuse("rope", "k must", k=f(2, 64))
    refuse("rope", "q must", q=f(2, 64, 4).transpose(1, 2))
    refuse("rope", "q_out", q_out=f(2, 3, 64))
    refuse("rope", "k_out", k_out=f(2, 1, 64).bfloat16())
    refuse("rope", "positions", positions=i(3, 1))
    refuse("rope", "positions", positions=i(2, 3).t())
    refuse("rope", "cos_sin", cos_sin=f(32, 9).t())
    refuse("rope", "axes has 3", axes=bytes(3))
    refuse("rope_store", "slot_map", slot_map=i(3))
    refuse("rope_store", "v must", v=f(2, 1, 64))
    refuse("rope_store", "expected 2 of 64", k_cache=f(5, 3, 8, 64), v_cache=f(5, 3, 8, 64))
    refuse("rope_store", "one layout", v_cache=f(5, 8, 2, 64).transpose(1, 2))
    refuse("attn_paged", "f32 or bf16", q=f(2, 4, 64).half())
    refuse("attn_paged", "q must", q=f(2, 8, 64)[:, ::2])
    refuse("attn_paged", "expected 2 of 64", k_cache=f(5, 2, 8, 32), v_cache=f(5, 2, 8, 32))
    refuse("attn_paged", "contiguous rows", k_cache=f(5, 2, 64, 8).transpose(2, 3), v_cache=f(5, 2, 64, 8).transpose(2, 3))
    refuse("attn_paged", "token_start", token_start=i(2))
    refuse("attn_paged", "output", output=f(2, 4, 32))
    refuse("attn_paged", "window", window=-1)
    # strided rows, other cache orders and a missing token_start are fine (refused for being on the host only)
    for change in (dict(q=f(2, 10, 64)[:, 3:7]), dict(k_cache=f(5, 8, 2, 64).transpose(1, 2), v_cache=f(5, 8, 2, 64).transpose(1, 2)),
                   dict(token_start=None), dict(output=f(4, 4, 64)[::2])):
        refuse("attn_paged", "must be a CUDA tensor", **change)


def test_binding_workspace_size(L):
    import torch

    import serving_gdn_decode_gb300 as gdn
    q, kc = torch.zeros(6, 8, 128, dtype=torch.bfloat16), torch.zeros(50, 2, 16, 128, dtype=torch.bfloat16)
    assert gdn.gdn_attn_workspace_size(q, kc, 4) == workspace_size(L)[1]
    with pytest.raises(nat.GdnError) as e:
        gdn.gdn_attn_workspace_size(q[..., :96].contiguous(), kc[..., :96], 4)
    assert e.value.status == nat.GDN_ERR_UNSUPPORTED


def test_fast_division_is_exact():
    """The kernels' division by a constant (paged_internal.h), on the edges of every quotient."""
    rng = np.random.default_rng(0)
    for d in [1, 2, 3, 5, 7, 8, 16, 24, 48, 64, 100, 1000, 1 << 16, (1 << 31) - 1, *rng.integers(1, 1 << 31, 200).tolist()]:
        s = 0
        while (1 << s) < d:
            s += 1
        m = (((1 << 32) * ((1 << s) - d)) // d + 1) & 0xffffffff
        n = np.concatenate([rng.integers(0, 1 << 31, 200), np.arange(0, 5) * d, np.arange(1, 5) * d - 1, [(1 << 31) - 1]])
        n = n[(n >= 0) & (n < 1 << 31)].astype(object)
        assert all((((x * m) >> 32) + x) >> s == x // d for x in n)
