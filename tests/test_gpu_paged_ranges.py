"""GPU tests of the full-attention operators over ranges that test_gpu_paged.py does not
reach, against plain implementations in 64 bits; its tolerances, and per request or row
where one request could hide another's error.
"""
import math

import pytest

from test_gpu_paged import ROPE_TOL, TOL, Case, clean_status, dtype_of, rel, table_of, torch  # noqa: F401 (fixtures among them)

pytestmark = pytest.mark.gpu

# Of a single row (64 elements or more): f32 as a whole tensor; bf16 by the largest rounding that all its elements
# could have at once, half a unit of the last of 8 bits.
ROW_TOL = {"f32": TOL["f32"], "bf16": 2.0 ** -8}


# ------------------------------------------------------------------ attention: long sums


@pytest.mark.parametrize("dim,group", [(64, 40), (128, 40), (256, 8), (128, 4)])
def test_attn_sums_of_long_items_do_not_drift(torch, dim, group):
    """A million keys per request and requests enough that none is split: 32 thousand tiles and more go into one
    running sum, and values of mean 1.5 show any leaning of its roundings.

    The one rounding of the result is below 2^-9 root-mean-square of an element, independent from column to column
    (each has a mean of its own): the mean signed error over `dim` columns stays below 4 * 2^-9 / sqrt(dim), four
    standard deviations.  f32 sums rounded to nearest add 2^-24 * sqrt(2^16) = 1.5e-5, which TOL holds."""
    import serving_gdn_decode_gb300 as gdn
    n, page, n_req = 1 << 20, 1024, 456
    g = torch.Generator(device="cuda").manual_seed(dim + group)
    rand = lambda f, *s: f(*s, device="cuda", generator=g)  # noqa: E731
    k = rand(torch.randn, n // page, 1, page, dim).to(torch.bfloat16)
    v = (1.0 + rand(torch.rand, dim) + 0.5 * (rand(torch.rand, n // page, 1, page, dim) - 0.5)).to(torch.bfloat16)
    q = rand(torch.randn, n_req, group, dim).to(torch.bfloat16)
    out = torch.empty_like(q)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].repeat(n_req, 1).contiguous()  # one cache for all
    lens = torch.full((n_req,), n, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.gdn_attn_workspace_size(q, k, n_req), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_paged(q, k, v, table, lens, None, out, ws)
    for r in (0, 201, n_req - 1):
        p = torch.softmax(q[r].double() @ k.reshape(-1, dim).double().T / math.sqrt(dim), -1)
        ref = p @ v.reshape(-1, dim).double()
        assert rel(out[r], ref) <= TOL["bf16"]
        signed = float(((out[r].double() - ref) / ref).mean())
        assert abs(signed) <= 4 * 2.0 ** -9 / math.sqrt(dim)


# ------------------------------------------------------------------ attention: pages behind a sliding window


@pytest.mark.parametrize("dtype,dim,group,wins", [("bf16", 64, 2, (1, 1, 1)), ("bf16", 128, 8, (1, 4, 7)), ("bf16", 256, 8, (1, 2, 3)),
                                                  ("f32", 64, 2, (1, 3, 1)), ("f32", 256, 4, (1, 1, 2))])
@pytest.mark.parametrize("page", [1, 8, 16, 24, 32, 48])
@pytest.mark.parametrize("window", [1, 20, 64, 300])
def test_attn_pages_behind_the_window_may_be_gone(torch, dtype, dim, group, wins, page, window):
    """A server gives back the pages that a sliding window has left: their table entries are no pages any more,
    at any place of the window's begin in a tile, and the rows and the status word are as with them."""
    for first_len in (49, 64, 337, 1000):
        lens = [first_len, first_len + 15, first_len + 22]
        c = Case(torch, dtype, lens, wins=list(wins), dim=dim, group=group, n_kv=1, page=page, seed=first_len)
        ref = c.reference(torch, window=window)
        for s, (n, w) in enumerate(zip(lens, wins)):
            gone = max(0, n - w + 1 - window) // page  # pages of which no row sees a key
            c.table[s, :gone] = -1 if s % 2 else 1 << 20
        got = c.run(torch, window=window)
        for row in range(sum(wins)):
            assert rel(got[row], ref[row]) <= ROW_TOL[dtype]


def test_attn_a_page_that_one_row_sees_must_be_there(torch):
    """Of the window's keys the first one's page is missing: only the first of three tokens sees it."""
    from serving_gdn_decode_gb300 import _native as nat
    c = Case(torch, "bf16", [100, 50], wins=[3, 1], dim=64, group=2, page=1)
    ref = c.reference(torch, window=20)
    c.table[0, 100 - 3 + 1 - 20] = -1
    got = c.run(torch, window=20)
    assert bool(got[:3].isnan().all()) and rel(got[3], ref[3]) <= TOL["bf16"]
    assert nat.gdn_device_status(reset=True) == nat.GDN_DEVICE_BAD_PAGE


# ------------------------------------------------------------------ attention: f32's largest values


@pytest.mark.parametrize("dim,group", [(64, 1), (64, 12), (128, 3), (256, 2)])
def test_attn_f32_largest_values(torch, dim, group):
    """Values and keys up to f32's largest are finite in their TF32 halves too: one key's value comes back (to
    2^-22), a key with the lowest value is as good as masked where the score says so."""
    c = Case(torch, "f32", [1, 3, 40], dim=dim, group=group, n_kv=1, page=4)
    top = torch.finfo(torch.float32).max
    p = int(c.table[0, 0])
    c.v[p, 0, 0, ::2], c.v[p, 0, 0, 1::2] = top, -top
    # request 1: q is positive in its first element only, keys 0 and 2 have f32's lowest there: scores of -1e35 and less
    row = c.q[1].zero_()
    row[:, 0] = 1e-3
    p = int(c.table[1, 0])
    c.k[p, 0, 0, 0], c.k[p, 0, 2, 0] = -top, -top
    c.k[p, 0, 1, 0] = 1.0
    c.v[p, 0, 0] = top / 2
    c.q_dev.copy_(c.q), c.k_dev.copy_(c.k), c.v_dev.copy_(c.v)
    got, ref = c.run(torch), c.reference(torch)
    for r in range(3):
        assert rel(got[r], ref[r]) <= TOL["f32"]


# ------------------------------------------------------------------ attention: wide rows, long and split; prompts among decodes


def check_rows(torch, c, dtype, **kw):
    ref, got = c.reference(torch, **kw), c.run(torch, **kw)
    for row in range(len(ref)):
        assert rel(got[row], ref[row]) <= ROW_TOL[dtype], row


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [24, 32])
@pytest.mark.parametrize("group,wins", [(16, (1, 1, 1)), (32, (1, 1, 1)), (40, (1, 1, 1)), (64, (1, 1, 1)), (8, (7, 1, 4))])
def test_attn_wide_rows_over_long_keys(torch, dtype, dim, page, group, wins):
    """Blocks of 16, 32 and 64 rows per key head whose items are split over many CTAs and joined, on pages that hold
    whole tiles and on pages that do not; every row by itself."""
    check_rows(torch, Case(torch, dtype, [5003, 64, 1711], wins=list(wins), dim=dim, group=group, n_kv=1, page=page), dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 8), (256, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_attn_prompts_among_decodes(torch, dtype, dim, group, window):
    """A step with whole prompts, the rest of one, and single tokens: many row blocks per request."""
    c = Case(torch, dtype, [150, 900, 333, 1, 70], wins=[150, 1, 41, 1, 70], dim=dim, group=group, n_kv=2, page=16)
    check_rows(torch, c, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 3), (64, 6), (64, 14), (128, 4), (128, 7), (128, 14), (256, 2), (256, 4), (256, 14)])
@pytest.mark.parametrize("page", [16, 24, 32])
def test_attn_unseen_values_of_wide_rows(torch, dtype, dim, group, page):
    """Windows of four tokens whose blocks of rows go over one, two and four warps: the newest key and value are NaN
    and infinite, and reach the newest token only; before the sliding window everything is."""
    window = 37
    c = Case(torch, dtype, [500, 93, 64], wins=[4, 4, 4], dim=dim, group=group, n_kv=1, page=page)
    ref = c.reference(torch, window=window)
    for s, n in enumerate(c.lens):
        for j in [*range(n - 4 + 1 - window), n - 1]:
            p = int(c.table[s, j // page])
            c.k[p, 0, j % page], c.v[p, 0, j % page] = math.inf if j % 2 else math.nan, math.nan if j % 2 else -math.inf
    c.k_dev.copy_(c.k), c.v_dev.copy_(c.v)
    got = c.run(torch, window=window)
    for row in range(12):
        if row % 4 == 3:
            assert not bool(got[row].isfinite().any())
        else:
            assert rel(got[row], ref[row]) <= ROW_TOL[dtype], row


# ------------------------------------------------------------------ rope: prompts


def rope_all(torch, x, pos, table, axes, inter, sign=1.0):
    """rope_reference of many tokens: all pairs at once, in 64 bits on the GPU."""
    half = table.shape[1] // 2
    at = pos.long()[torch.tensor(list(axes), device="cuda")].T  # [tokens, pairs]
    j = torch.arange(half, device="cuda")
    c, s = table[at, j].double()[:, None], sign * table[at, half + j].double()[:, None]
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if inter else (slice(0, half), slice(half, 2 * half))
    y = x.double().clone()
    y[..., a] = x[..., a].double() * c - x[..., b].double() * s
    y[..., b] = x[..., b].double() * c + x[..., a].double() * s
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [4001, 20011])  # one to a few parts per token, several steps of rows each
@pytest.mark.parametrize("n_q,n_kv,dim,rot,axes,inter", [(32, 8, 128, 128, 3, False), (7, 1, 64, 64, 2, False), (16, 2, 256, 64, 1, True),
                                                       (5, 3, 128, 128, 2, True), (3, 1, 256, 256, 1, False), (6, 2, 72, 72, 2, False),
                                                       (9, 3, 34, 20, 2, False)])
def test_rope_and_store_of_prompts(torch, dtype, n, n_q, n_kv, dim, rot, axes, inter):
    """Every form of both kernels over prompts: the store into a paged cache with q in place in the fused rows, and
    the rotation there and back."""
    import serving_gdn_decode_gb300 as gdn
    dt, page = dtype_of(torch, dtype), 16
    g = torch.Generator(device="cuda").manual_seed(n + dim)
    rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(dt)  # noqa: E731
    fused = rand(n, (n_q + 2 * n_kv) * dim)
    q, k, v = (x.unflatten(1, (-1, dim)) for x in fused.split([n_q * dim, n_kv * dim, n_kv * dim], 1))
    table = table_of(torch, 500, rot).cuda()
    pos = torch.randint(0, 500, (axes, n), device="cuda", generator=g).to(torch.int32)
    of_pair = bytes(j * axes // (rot // 2) for j in range(rot // 2))
    pages = n // page + 2
    kc, vc = rand(pages, n_kv, page, dim), rand(pages, n_kv, page, dim)
    slots = torch.randperm(pages * page, device="cuda", generator=g)[:n].to(torch.int32)
    slots[::61] = -1
    before = [x.clone() for x in (q, k, v, kc, vc)]
    tol = ROPE_TOL[dtype]

    qo, ko = torch.empty_like(before[0]), torch.empty_like(before[1])
    gdn.gdn_rope(q, k, pos, table, qo, ko, axes=of_pair, interleaved=inter)
    for got, x in ((qo, before[0]), (ko, before[1])):
        want = rope_all(torch, x, pos, table, of_pair, inter)
        assert rel(got, want) <= tol and torch.equal(got[..., rot:], x[..., rot:])
        per_token = (got.double() - want).flatten(1).norm(dim=1) / want.flatten(1).norm(dim=1)
        assert float(per_token.max()) <= 2.5 * tol  # of a token's elements alone: bf16's largest roundings are twice its usual ones
    gdn.gdn_rope(qo, ko, pos, table, qo, ko, axes=of_pair, interleaved=inter, inverse=True)
    assert rel(qo, before[0]) <= 2 * tol and rel(ko, before[1]) <= 2 * tol

    gdn.gdn_rope_store(q, k, v, pos, table, slots, kc, vc, q, axes=of_pair, interleaved=inter)
    assert rel(q, rope_all(torch, before[0], pos, table, of_pair, inter)) <= tol
    assert torch.equal(k, before[1]) and torch.equal(v, before[2])
    flat = lambda x: x.transpose(1, 2).reshape(-1, n_kv, dim)  # noqa: E731
    has = slots >= 0
    at = slots[has].long()
    assert torch.equal(flat(vc)[at], before[2][has])
    assert rel(flat(kc)[at], rope_all(torch, before[1], pos, table, of_pair, inter)[has]) <= tol
    rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(flat(kc)[rest], flat(before[3])[rest]) and torch.equal(flat(vc)[rest], flat(before[4])[rest])


# ------------------------------------------------------------------ the example


@pytest.mark.parametrize("steps", [0, 1, 2])
def test_hybrid_example_of_few_steps(torch, capsys, steps):
    """Without a decode step the logits are the prompts'; with one, nothing is captured yet.  The bound is
    test_hybrid_example's."""
    from serving_gdn_decode_gb300 import hybrid_step
    args = ["--requests", "3", "--prompt", "17", "--steps", str(steps), "--check"]
    assert hybrid_step.main(args) <= 1e-3
    assert "device status 0" in capsys.readouterr().out
