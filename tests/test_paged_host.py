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


def test_binding_refuses_before_calling():
    import torch

    import serving_gdn_decode_gb300 as gdn
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q, kc, out = torch.zeros(2, 4, 64), torch.zeros(5, 2, 8, 64), torch.zeros(2, 4, 64)
    with pytest.raises(nat.GdnError, match="must be a CUDA tensor"):
        gdn.gdn_attn_paged(q, kc, kc, i(2, 3), i(2), None, out, torch.zeros(10))
    with pytest.raises(nat.GdnError, match="must be a CUDA tensor"):
        gdn.gdn_rope(q, q, i(2), torch.zeros(9, 64), out, out)
    with pytest.raises(TypeError, match="slot_map"):
        gdn.gdn_rope_store(q, q, q, i(2), torch.zeros(9, 64), [0, 1], kc, kc, out)
    with pytest.raises(TypeError, match="n_free"):
        gdn.gdn_kv_plan(i(2), i(2), i(2), i(4), 4, i(2, 3), 8, 5, i(2), i(2), i(1), i(3), i(2), i(2))


def test_binding_shape_rules():
    """The marshalling's own checks, on host tensors (which the calls refuse)."""
    import torch

    from serving_gdn_decode_gb300 import paged
    q, kc = torch.zeros(2, 4, 64), torch.zeros(5, 2, 8, 64)
    p = paged._attn_params(q, kc, kc, 3, 7, None, None, 9)
    assert (p.head_dim, p.n_q_heads, p.n_kv_heads, p.page_size, p.n_pages, p.max_pages, p.window) == (64, 4, 2, 8, 5, 7, 9)
    assert (p.cache_page_stride, p.cache_head_stride, p.cache_slot_stride) == (1024, 512, 64)
    assert p.scale == pytest.approx(0.125) and (p.q_stride, p.out_stride) == (256, 256)
    nhd = torch.zeros(5, 8, 2, 64).transpose(1, 2)
    p = paged._attn_params(q, nhd, nhd, 3, 7, None, 0.5, 0)
    assert (p.cache_page_stride, p.cache_head_stride, p.cache_slot_stride, p.scale) == (1024, 64, 128, 0.5)
    wide = torch.zeros(2, 10, 64)[:, 3:7]
    assert paged._attn_params(wide, kc, kc, 1, 1, None, None, 0).q_stride == 640
    for bad in (torch.zeros(2, 64, 4).transpose(1, 2), torch.zeros(2, 8, 64)[:, ::2], torch.zeros(4, 64)):
        with pytest.raises(nat.GdnError):
            paged._attn_params(bad, kc, kc, 1, 1, None, None, 0)
    with pytest.raises(nat.GdnError, match="f32 or bf16"):
        paged._attn_params(q.half(), kc, kc, 1, 1, None, None, 0)
    with pytest.raises(nat.GdnError, match="k_cache"):
        paged._attn_params(q.bfloat16(), kc, kc, 1, 1, None, None, 0)
    with pytest.raises(nat.GdnError, match="one layout"):
        paged._attn_params(q, kc, nhd, 1, 1, None, None, 0)
    with pytest.raises(nat.GdnError, match="expected 2 of 64"):
        paged._attn_params(q, torch.zeros(5, 2, 8, 128), torch.zeros(5, 2, 8, 128), 1, 1, None, None, 0)
    k, pos, cs = torch.zeros(2, 2, 64), torch.zeros(3, 2, dtype=torch.int32), torch.zeros(9, 32)
    p = paged._rope_params(q, k, None, pos, cs, q, k, None, None, None, bytes([2] * 16), 1)
    assert (p.n_axes, p.positions_stride, p.rot_dim, p.n_positions, p.flags, p.axis_of_pair[15]) == (3, 2, 32, 9, 1, 2)
    for change, text in ((dict(axes=bytes(3)), "axes has 3"), (dict(positions=pos.long()), "positions"),
                         (dict(positions=pos[:, :1]), "positions"), (dict(cos_sin=cs.double()), "cos_sin"),
                         (dict(cos_sin=cs.t()), "cos_sin"), (dict(q_out=torch.zeros(2, 3, 64)), "q_out"),
                         (dict(k_out=k.bfloat16()), "k_out")):
        a = dict(q=q, k=k, v=None, positions=pos, cos_sin=cs, q_out=q, k_out=k, slot_map=None, k_cache=None,
                 v_cache=None, axes=bytes(16), flags=0)
        a.update(change)
        with pytest.raises(nat.GdnError, match=text):
            paged._rope_params(**a)


def test_kept_params_are_bounded(monkeypatch):
    """The kept structs depend on shapes only and cannot grow without end."""
    from serving_gdn_decode_gb300 import paged
    monkeypatch.setattr(paged, "_kept", {})
    monkeypatch.setattr(paged, "_MAX_KEPT", 8)
    for i in range(50):
        assert paged._keep(i, lambda: i) == i
        assert paged._keep(i, lambda: -1) == i
        assert len(paged._kept) <= 8


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
