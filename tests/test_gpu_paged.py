"""GPU tests of the full-attention operators (gdn_kv_plan, gdn_rope,
gdn_rope_store, gdn_attn_paged) against plain implementations in 64 bits.

Tolerances, from the arithmetic:
* f32 attention: an operand is hi + lo in TF32 up to 2^-22 of it and the lo * lo
  product is left out, so a product is off by 3 * 2^-22 of |q||k| at most.  With
  sum |q k| * scale below 24 for these inputs, a score is off by 1.8e-5 and a
  probability, like the output, by at most twice that: 4e-5 at the very worst,
  were all errors of one sign.  Their signs are random over 64 to 256 products,
  so 2e-5 is ample.
* bf16 attention: the same sums, then one rounding to nearest of each element: off
  by 2^-8 of it at most, uniformly, so 2^-8 / sqrt(3) = 2.3e-3 root-mean-square for
  elements just above a power of two and half of that just below the next; 1.7e-3
  over all: rel-L2 2^-9 + 2e-5, which these tests' thousands of elements stay below.
* rope: two f32 products and a sum, 3 * 2^-24 of sqrt(a^2 + b^2): rel-L2 2e-7;
  bf16 adds its one rounding, 2^-9 as above.
* whole numbers (the plan; copies of v): equal.
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TOL = {"f32": 2e-5, "bf16": 2.0 ** -9 + 2e-5}


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a CUDA device"
    from serving_gdn_decode_gb300 import build
    build.build()
    return t


@pytest.fixture(autouse=True)
def clean_status(torch):
    """Every test leaves the device status word clear, unless it reads it itself."""
    from serving_gdn_decode_gb300 import _native as nat
    nat.gdn_device_status(reset=True)
    yield
    assert nat.gdn_device_status(reset=True) == 0


def status():
    from serving_gdn_decode_gb300 import _native as nat
    return nat.gdn_device_status(reset=True)


def dtype_of(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def rel(got, ref):
    got, ref = got.double().cpu(), ref.double().cpu()
    assert bool(got.isfinite().all())
    return float((got - ref).norm() / ref.norm()) if float(ref.norm()) else float(got.norm())


# ------------------------------------------------------------------ attention


class Case:
    """A paged cache with requests in it.  Slots that no request holds are NaN."""

    def __init__(self, torch, dtype, lens, wins=None, n_kv=2, group=2, dim=128, page=16, layout="hnd", seed=0,
                 extra=3, max_pages=None, fused_q=False):
        g = torch.Generator().manual_seed(seed)
        dt = dtype_of(torch, dtype)
        self.lens, self.wins = list(lens), list(wins) if wins is not None else [1] * len(lens)
        self.n_kv, self.group, self.dim, self.page = n_kv, group, dim, page
        pages = [-(-n // page) for n in self.lens]
        n_pages = sum(pages) + extra
        order = torch.randperm(n_pages, generator=g).tolist()
        width = max(max(pages), 1) if max_pages is None else max_pages
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        k = torch.full((n_pages, n_kv, page, dim), math.nan)
        v = torch.full((n_pages, n_kv, page, dim), math.nan)
        at = 0
        for s, n in enumerate(self.lens):
            for j in range(pages[s]):
                table[s, j] = order[at]
                fill = min(page, n - j * page)
                k[order[at], :, :fill] = torch.randn(n_kv, fill, dim, generator=g)
                v[order[at], :, :fill] = torch.randn(n_kv, fill, dim, generator=g)
                at += 1
        self.k, self.v = k.to(dt), v.to(dt)
        n = sum(self.wins)
        q = (1.5 * torch.randn(n, n_kv * group, dim, generator=g)).to(dt)
        self.q = q
        self.table = table.cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.start = torch.tensor([0] + list(np.cumsum(self.wins)), dtype=torch.int32).cuda()
        self.k_dev, self.v_dev = self.k.cuda(), self.v.cuda()
        if layout == "nhd":  # [page, slot, head, dim] in memory
            self.k_dev = self.k_dev.transpose(1, 2).contiguous().transpose(1, 2)
            self.v_dev = self.v_dev.transpose(1, 2).contiguous().transpose(1, 2)
        elif layout == "both":  # K and V of a page side by side
            both = torch.stack([self.k_dev, self.v_dev], 1).contiguous()
            self.k_dev, self.v_dev = both[:, 0], both[:, 1]
        self.q_dev = q.cuda()
        if fused_q:  # rows of a wider projection
            wide = torch.zeros(n, (n_kv * group + 2 * n_kv) * dim, dtype=dt, device="cuda")
            view = wide[:, : n_kv * group * dim].unflatten(1, (n_kv * group, dim))
            view.copy_(self.q_dev)
            self.q_dev = view
        self.out = torch.full((n, n_kv * group, dim), 7.0, dtype=dt, device="cuda")

    def run(self, torch, scale=None, window=0, stream=None, start=True):
        import serving_gdn_decode_gb300 as gdn
        size = gdn.gdn_attn_workspace_size(self.q_dev, self.k_dev, len(self.lens))
        # whatever the workspace holds must not matter
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        gdn.gdn_attn_paged(self.q_dev, self.k_dev, self.v_dev, self.table, self.kv_lens,
                           self.start if start else None, self.out, ws, scale=scale, window=window,
                           stream=stream)
        torch.cuda.synchronize()
        return self.out

    def reference(self, torch, scale=None, window=0):
        scale = 1.0 / math.sqrt(self.dim) if scale is None else scale
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        row = 0
        for s, (n, w) in enumerate(zip(self.lens, self.wins)):
            pages = self.table[s, : -(-n // self.page)].long().cpu()
            k = self.k[pages].double().permute(1, 0, 2, 3).reshape(self.n_kv, -1, self.dim)
            v = self.v[pages].double().permute(1, 0, 2, 3).reshape(self.n_kv, -1, self.dim)
            for t in range(w):
                hi = n - w + t + 1
                lo = max(0, hi - window) if window else 0
                if hi > 0:
                    q = self.q[row].double().view(self.n_kv, self.group, self.dim)
                    p = torch.softmax(scale * torch.einsum("hgd,hkd->hgk", q, k[:, lo:hi]), -1)
                    out[row] = torch.einsum("hgk,hkd->hgd", p, v[:, lo:hi]).reshape(-1, self.dim)
                row += 1
        return out

    def check(self, torch, dtype, **kw):
        ref = self.reference(torch, **{k: v for k, v in kw.items() if k in ("scale", "window")})
        got = self.run(torch, **kw)
        assert rel(got, ref) <= TOL[dtype]
        # rows without a key are exactly zero
        empty = (ref == 0).all(-1).all(-1)
        assert not got[empty.to(got.device)].any()


EDGES = [1, 0, 15, 16, 17, 63, 64, 65, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_attn_lengths(torch, dtype, dim, group):
    Case(torch, dtype, EDGES, dim=dim, group=group, n_kv=2).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [9, 16, 17, 40])
def test_attn_large_groups(torch, dtype, group):
    """More query heads per key head than one row tile takes, up to several row blocks."""
    Case(torch, dtype, [200, 1, 77], dim=64, group=group, n_kv=1).check(torch, dtype)
    Case(torch, dtype, [70, 5], dim=256, group=group, n_kv=2).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 200])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
def test_attn_pages_and_layouts(torch, dtype, page, layout):
    Case(torch, dtype, [130, 33, 0, 1], page=page, layout=layout).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 2), (128, 5), (256, 8)])
def test_attn_windows_of_tokens(torch, dtype, dim, group):
    """Ragged windows: several tokens per request, requests without any, more tokens than keys."""
    c = Case(torch, dtype, [4, 70, 64, 131, 9, 0, 2, 500], wins=[4, 3, 1, 7, 0, 0, 5, 16], dim=dim, group=group,
             n_kv=2)
    c.check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 1 << 30, (1 << 32) - 1])
def test_attn_sliding_window(torch, dtype, window):
    c = Case(torch, dtype, [1, 90, 64, 200, 333, 0], wins=[1, 1, 3, 6, 2, 0], dim=64, group=2)
    c.check(torch, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_unseen_nan_and_infinity(torch, dtype):
    """Keys and values that a row does not see -- before its window, after its own token -- may be anything."""
    c = Case(torch, dtype, [100, 40], wins=[4, 3], dim=128, group=2, page=16)
    window = 20
    bad = [(0, j) for j in range(0, 77)] + [(1, j) for j in range(0, 18)]
    for s, j in bad:  # before every row's window
        p = int(c.table[s, j // 16])
        c.k[p, :, j % 16], c.v[p, :, j % 16] = math.inf, math.nan
    ref = c.reference(torch, window=window)
    # the newest key of request 0, seen by its last row only
    p = int(c.table[0, 99 // 16])
    c.k[p, :, 99 % 16, 0] = math.nan
    c.v[p, :, 99 % 16] = -math.inf
    c.k_dev.copy_(c.k)
    c.v_dev.copy_(c.v)
    got = c.run(torch, window=window)
    keep = [0, 1, 2, 4, 5, 6]
    assert rel(got[keep], ref[keep]) <= TOL[dtype]
    assert bool(got[3].isnan().all())


def test_attn_scores_of_minus_infinity(torch):
    """A visible score of -inf has weight zero; a row whose visible scores are all -inf is 0 / 0."""
    c = Case(torch, "f32", [40, 3], dim=64, group=1, n_kv=1)
    c.q[:] = 1.0
    c.k[:] = torch.where(c.k.isnan(), c.k, c.k.abs())
    ref = c.reference(torch)
    c.q_dev.copy_(c.q)
    for j in range(3):
        p = int(c.table[1, 0])
        c.k[p, :, j] = -1e38
    c.k_dev.copy_(c.k)
    got = c.run(torch, scale=1.0 / 8)
    assert rel(got[:1], ref[:1]) <= TOL["f32"]
    big = c.run(torch, scale=1e30)  # overflows to -inf in f32
    assert bool(big[1].isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_long_and_split(torch, dtype):
    """One long request is split over the whole GPU and joined; with others beside it."""
    Case(torch, dtype, [20011], dim=128, group=4, n_kv=1, page=16).check(torch, dtype)
    Case(torch, dtype, [9000, 1, 0, 65, 3000, 64], wins=[2, 1, 0, 1, 4, 1], dim=64, group=3, n_kv=2,
         page=32).check(torch, dtype)


def test_attn_many_requests(torch):
    """More requests than threads of a CTA, some idle."""
    lens = [(37 * i) % 150 if i % 7 else 0 for i in range(700)]
    Case(torch, "bf16", lens, wins=[1 if n else 0 for n in lens], dim=64, group=2, n_kv=1).check(torch, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_pages", [8, 16, 17, 100])
def test_attn_table_width(torch, dtype, max_pages):
    """A table that bounds the lengths keeps an item in one CTA, a wider one lets it be split: either is right,
    with more items than CTAs and with fewer."""
    lens = [(13 * i) % 129 for i in range(90)]
    for n, n_kv in ((90, 7), (3, 1)):
        Case(torch, dtype, lens[:n], wins=[min(3, k) for k in lens[:n]], n_kv=n_kv, group=2, dim=64, page=16,
             max_pages=max_pages).check(torch, dtype)
    Case(torch, dtype, [128, 5, 0, 64], dim=256, group=9, n_kv=2, max_pages=max_pages).check(torch, dtype, window=40)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attn_scales(torch, scale):
    Case(torch, "f32", [100, 17], dim=64).check(torch, "f32", scale=scale)


def test_attn_peaked(torch):
    """Scores hundreds apart: the running maximum moves far, and no sum overflows."""
    c = Case(torch, "f32", [1000], dim=64, group=2, n_kv=1)
    c.q *= 40
    c.q_dev.copy_(c.q)
    ref, got = c.reference(torch), c.run(torch)
    # a score s is off by s * 2^-22 * 3, up to 1000 * 7e-7
    assert rel(got, ref) <= 2e-3


def test_attn_strided_q_other_stream_and_runs(torch):
    c = Case(torch, "bf16", [300, 40, 5000], dim=128, group=4, fused_q=True)
    side = torch.cuda.Stream()
    first = c.run(torch, stream=side).clone()
    assert rel(first, c.reference(torch)) <= TOL["bf16"]
    c.out.fill_(3.0)
    assert torch.equal(c.run(torch), first)  # the same bits on every run
    c.out.fill_(3.0)
    assert torch.equal(c.run(torch, start=False), first)  # one token per request: no offsets needed


def test_attn_does_not_depend_on_the_batch(torch):
    """A request alone and among others, split or not, agrees to the tolerance."""
    lens = [700, 64, 1300]
    c = Case(torch, "f32", lens, dim=128, group=2)
    got = c.run(torch).clone()
    for s in range(3):
        d = Case(torch, "f32", lens, dim=128, group=2)
        d.kv_lens[:] = 0
        d.kv_lens[s] = lens[s]
        assert rel(d.run(torch)[s], got[s]) <= TOL["f32"]


def test_attn_writes_its_rows_only(torch):
    import serving_gdn_decode_gb300 as gdn
    c = Case(torch, "bf16", [90, 0, 33], wins=[2, 0, 1], dim=64, group=2)
    size = gdn.gdn_attn_workspace_size(c.q_dev, c.k_dev, 3)
    ws = torch.full((size + 512,), 9, dtype=torch.uint8, device="cuda")
    wide = torch.full((5, 3 * 4 * 64), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[1:4, : 4 * 64].unflatten(1, (4, 64))
    gdn.gdn_attn_paged(c.q_dev, c.k_dev, c.v_dev, c.table, c.kv_lens, c.start, out, ws[256: 256 + size])
    torch.cuda.synchronize()
    assert rel(out, c.reference(torch)) <= TOL["bf16"]
    assert bool((ws[:256] == 9).all()) and bool((ws[256 + size:] == 9).all())
    assert bool((wide[0] == 5).all()) and bool((wide[4] == 5).all()) and bool((wide[:, 256:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_output_aligned_to_an_element_only(torch, dtype):
    c = Case(torch, dtype, [90, 500, 3000], dim=64, group=3)
    raw = torch.full((c.out.numel() + 2,), 5.0, dtype=c.out.dtype, device="cuda")
    c.out = raw[1:-1].view(c.out.shape)
    c.check(torch, dtype)
    assert float(raw[0]) == 5 and float(raw[-1]) == 5


def test_attn_offsets_past_32_bits(torch):
    """A cache of more than 2^32 elements: pages at its very end."""
    import serving_gdn_decode_gb300 as gdn
    page, n_kv, dim = 64, 8, 128
    n_pages = (1 << 32) // (page * n_kv * dim) + 8
    k = torch.empty(n_pages, n_kv, page, dim, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(3)
    used = [n_pages - 1, 5, n_pages - 3]
    for p in used:
        k[p] = torch.randn(n_kv, page, dim, device="cuda", generator=g).to(torch.bfloat16)
        v[p] = torch.randn(n_kv, page, dim, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(1, n_kv * 2, dim, device="cuda", generator=g).to(torch.bfloat16)
    n = 2 * page + 17
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q)
    ws = torch.empty(gdn.gdn_attn_workspace_size(q, k, 1), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_paged(q, k, v, table, lens, None, out, ws)
    kk, vv = (x[used].double().permute(1, 0, 2, 3).reshape(n_kv, -1, dim)[:, :n] for x in (k, v))
    p = torch.softmax(torch.einsum("hgd,hkd->hgk", q[0].double().view(n_kv, 2, dim), kk) / math.sqrt(dim), -1)
    ref = torch.einsum("hgk,hkd->hgd", p, vv).reshape(1, -1, dim)
    assert rel(out, ref) <= TOL["bf16"]
    # the store finds the same places
    slot = torch.tensor([(n_pages - 1) * page + 63], dtype=torch.int32, device="cuda")
    cs = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], 1).cuda()
    kn = torch.randn(1, n_kv, dim, device="cuda", generator=g).to(torch.bfloat16)
    gdn.gdn_rope_store(q, kn, kn, torch.zeros(1, dtype=torch.int32, device="cuda"), cs, slot, k, v, torch.empty_like(q))
    assert torch.equal(k[n_pages - 1, :, 63], kn[0]) and torch.equal(v[n_pages - 1, :, 63], kn[0])


def test_attn_bad_data_is_reported(torch):
    """Numbers that cannot be followed are clipped, the rows concerned are NaN or left out, and the status says so."""
    from serving_gdn_decode_gb300 import _native as nat
    c = Case(torch, "bf16", [100, 40, 30], dim=64, group=2)
    ref = c.reference(torch)
    c.table[0, 3] = 1 << 20
    got = c.run(torch)
    assert bool(got[0].isnan().all()) and rel(got[1:], ref[1:]) <= TOL["bf16"]
    assert status() == nat.GDN_DEVICE_BAD_PAGE
    c = Case(torch, "bf16", [100, 40, 112], dim=64, group=2)
    ref = c.reference(torch)
    c.kv_lens[0], c.kv_lens[1], c.kv_lens[2] = 100, -5, 1 << 30
    got = c.run(torch)
    assert rel(got[0], ref[0]) <= TOL["bf16"] and not got[1].any() and rel(got[2], ref[2]) <= TOL["bf16"]
    assert status() == nat.GDN_DEVICE_BAD_REQUEST
    c = Case(torch, "bf16", [100, 40, 112], dim=64, group=2)
    c.start[3] = 1000
    got = c.run(torch)
    assert rel(got, c.reference(torch)) <= TOL["bf16"]
    assert status() == nat.GDN_DEVICE_BAD_REQUEST


# ------------------------------------------------------------------ rope


def table_of(torch, rows, rot):
    freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def rope_reference(torch, x, pos, table, axes, inter, sign=1.0):
    y = x.double().clone()
    half = table.shape[1] // 2
    for j in range(half):
        at = pos[axes[j]].long()
        c, s = table[at, j].double()[:, None], sign * table[at, half + j].double()[:, None]
        a, b = (2 * j, 2 * j + 1) if inter else (j, j + half)
        y[..., a] = x[..., a].double() * c - x[..., b].double() * s
        y[..., b] = x[..., b].double() * c + x[..., a].double() * s
    return y


ROPE_TOL = {"f32": 2e-7, "bf16": 2.0 ** -9}


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,rot,n_q,n_kv,n_axes", [
    (128, 128, 4, 2, 3), (256, 64, 16, 1, 2), (64, 64, 3, 3, 1), (64, 20, 5, 1, 4), (6, 2, 1, 1, 1), (80, 80, 2, 2, 2),
    (256, 256, 40, 8, 4), (34, 34, 2, 1, 3), (32, 32, 7, 2, 2), (16, 16, 1, 1, 1), (72, 72, 5, 5, 2)])
def test_rope_and_inverse(torch, dtype, inter, dim, rot, n_q, n_kv, n_axes):
    import serving_gdn_decode_gb300 as gdn
    dt, n = dtype_of(torch, dtype), 37
    g = torch.Generator().manual_seed(dim + rot)
    q, k = (torch.randn(n, h, dim, generator=g).to(dt) for h in (n_q, n_kv))
    table = table_of(torch, 500, rot)
    pos = torch.randint(0, 500, (n_axes, n), generator=g, dtype=torch.int32)
    axes = bytes(j % n_axes for j in range(rot // 2))
    for sign, inverse in ((1.0, False), (-1.0, True)):
        qo, ko = torch.zeros_like(q).cuda(), torch.zeros_like(k).cuda()
        gdn.gdn_rope(q.cuda(), k.cuda(), pos.cuda(), table.cuda(), qo, ko, axes=axes, interleaved=inter,
                     inverse=inverse)
        for got, x in ((qo, q), (ko, k)):
            ref = rope_reference(torch, x, pos, table, axes, inter, sign)
            assert rel(got, ref) <= ROPE_TOL[dtype]
            assert torch.equal(got[..., rot:].cpu(), x[..., rot:])


def test_rope_gradient_against_differences(torch):
    """The inverse rotation of the output's gradient is the gradient: against central differences of
    L = sum(w * rope(x)), linear in x, so that the difference quotient is exact up to f32 rounding."""
    import serving_gdn_decode_gb300 as gdn
    n, h, d = 5, 2, 16
    g = torch.Generator().manual_seed(9)
    x, w = torch.randn(n, h, d, generator=g), torch.randn(n, h, d, generator=g)
    table, pos = table_of(torch, 64, d).cuda(), torch.randint(0, 64, (n,), generator=g, dtype=torch.int32).cuda()

    def rope(a, inverse=False):
        a = a.float().cuda()
        o, k = torch.empty_like(a), torch.empty_like(a)
        gdn.gdn_rope(a, a.clone(), pos, table, o, k, inverse=inverse)
        return o.double().cpu()

    grad = rope(w, inverse=True)
    eps = 0.5  # L is linear: a wide step loses nothing
    for at in [(0, 0, 0), (2, 1, 7), (4, 0, 8), (3, 1, 15)]:
        up, down = x.double().clone(), x.double().clone()
        up[at] += eps
        down[at] -= eps
        slope = float((w.double() * (rope(up) - rope(down))).sum()) / (2 * eps)
        # each rope value is off by 2^-23 of about 4, 32 of them with weights of about 1
        assert abs(slope - float(grad[at])) <= 3e-5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["hnd", "nhd"])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_rope_store(torch, dtype, layout, n):
    """Views of a fused projection; padding tokens without a slot; the rest of the cache untouched."""
    import serving_gdn_decode_gb300 as gdn
    dt, n_q, n_kv, dim, page = dtype_of(torch, dtype), 6, 2, 64, 12
    g = torch.Generator().manual_seed(n)
    qkv = torch.randn(n, (n_q + 2 * n_kv) * dim, generator=g).to(dt)
    fused = qkv.cuda()
    q, k, v = (x.unflatten(1, (-1, dim)) for x in fused.split([n_q * dim, n_kv * dim, n_kv * dim], 1))
    pages = n // page + 4
    shape = (pages, n_kv, page, dim)
    kc, vc = torch.randn(shape, generator=g).to(dt), torch.randn(shape, generator=g).to(dt)
    kd, vd = kc.cuda(), vc.cuda()
    if layout == "nhd":
        kd, vd = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (kd, vd))
    slots = torch.randperm(pages * page, generator=g)[:n].to(torch.int32)
    slots[n // 2] = -1 if n > 1 else slots[0]
    pos = torch.randint(0, 90, (2, n), generator=g, dtype=torch.int32)
    table, axes = table_of(torch, 90, 32), bytes([0, 1] * 8)
    host = [x.cpu().clone() for x in (q, k, v)]
    # q rotated in place, in the fused rows
    gdn.gdn_rope_store(q, k, v, pos.cuda(), table.cuda(), slots.cuda(), kd, vd, q, axes=axes)
    assert rel(q, rope_reference(torch, host[0], pos, table, axes, False)) <= ROPE_TOL[dtype]
    assert torch.equal(k.cpu(), host[1]) and torch.equal(v.cpu(), host[2])
    kr = rope_reference(torch, host[1], pos, table, axes, False)
    want_k, want_v = kc.double(), vc.clone()
    for i, s in enumerate(slots.tolist()):
        if s >= 0:
            want_k[s // page, :, s % page] = kr[i]
            want_v[s // page, :, s % page] = host[2][i]
    assert torch.equal(vd.cpu(), want_v)
    assert rel(kd, want_k) <= ROPE_TOL[dtype]
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[slots[slots >= 0].long()] = False
    flat = lambda x: x.transpose(1, 2).reshape(-1, n_kv, dim)  # noqa: E731
    assert torch.equal(flat(kd.cpu())[untouched], flat(kc)[untouched])


def test_rope_unaligned_and_in_place(torch):
    """Rows that no 16-byte access fits, in place, on another stream."""
    import serving_gdn_decode_gb300 as gdn
    g = torch.Generator().manual_seed(1)
    n, dim = 9, 32
    raw = torch.randn(n * (3 * dim + 3) + 1, generator=g).to(torch.bfloat16).cuda()
    rows = raw[1:].view(n, 3 * dim + 3)
    q, k = rows[:, : 2 * dim].unflatten(1, (2, dim)), rows[:, 2 * dim: 3 * dim].unflatten(1, (1, dim))
    hq, hk, tail = q.cpu().clone(), k.cpu().clone(), rows[:, 3 * dim:].clone()
    pos = torch.arange(n, dtype=torch.int32)
    table = table_of(torch, n, dim)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pd, td = pos.cuda(), table.cuda()
    torch.cuda.synchronize()
    gdn.gdn_rope(q, k, pd, td, q, k, stream=side)
    side.synchronize()
    axes = [0] * (dim // 2)
    assert rel(q, rope_reference(torch, hq, pos[None], table, axes, False)) <= ROPE_TOL["bf16"]
    assert rel(k, rope_reference(torch, hk, pos[None], table, axes, False)) <= ROPE_TOL["bf16"]
    assert torch.equal(rows[:, 3 * dim:], tail)


def test_rope_bad_data_is_reported(torch):
    import serving_gdn_decode_gb300 as gdn
    from serving_gdn_decode_gb300 import _native as nat
    n, dim, page = 3, 64, 8
    q = torch.ones(n, 2, dim, device="cuda")
    k = torch.ones(n, 1, dim, device="cuda")
    kc, vc = torch.zeros(2, 1, page, dim, device="cuda"), torch.zeros(2, 1, page, dim, device="cuda")
    table = table_of(torch, 10, 32).cuda()
    pos = torch.tensor([1, 10, -1], dtype=torch.int32, device="cuda")
    slots = torch.tensor([3, 16, 1 << 30], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    gdn.gdn_rope_store(q, k, k, pos, table, slots, kc, vc, out)
    assert status() == nat.GDN_DEVICE_BAD_PAGE | nat.GDN_DEVICE_BAD_POSITION
    assert bool(out[0].isfinite().all()) and bool(out[1:, :, :32].isnan().all()) and bool((out[1:, :, 32:] == 1).all())
    assert int((vc != 0).sum()) == dim and bool((vc[0, 0, 3] == 1).all())


def test_rope_no_tokens(torch):
    import serving_gdn_decode_gb300 as gdn
    q = torch.zeros(0, 2, 64, device="cuda")
    gdn.gdn_rope(q, q, torch.zeros(0, dtype=torch.int32, device="cuda"), table_of(torch, 4, 64).cuda(), q, q)


# ------------------------------------------------------------------ plan


def plan_reference(ctx, new, owned, free, table, page, max_pages, n_slots):
    """One request after another, with a list for the stack."""
    free, table = list(free), [list(r) for r in table]
    kv, own, start, slots, pos = [], [], [0], [], []
    taken = short = False
    left = len(free)
    closed = False
    for s, (c, n, o) in enumerate(zip(ctx, new, owned)):
        need = max(o, -(-(c + n) // page))
        ok = need <= max_pages
        if ok and need > o:
            if closed or need - o > left:
                ok, closed, short = False, True, True
            else:
                for j in range(o, need):
                    table[s][j] = free.pop()
                left -= need - o
        kv.append(c + n if ok else c)
        own.append(need if ok else o)
        for i in range(n):
            pos.append(c + i)
            slots.append(table[s][(c + i) // page] * page + (c + i) % page if ok else -1)
        start.append(start[-1] + n)
    slots += [-1] * (n_slots - len(slots))
    pos += [0] * (n_slots - len(pos))
    return table, kv, own, [left], start, slots[:n_slots], pos[:n_slots], short


def plan_call(torch, ctx, new, owned, free, table, page, n_pages, n_slots, n_free=None):
    import serving_gdn_decode_gb300 as gdn
    i = lambda x: torch.tensor(np.asarray(x, dtype=np.int64), dtype=torch.int32).cuda()  # noqa: E731
    n = len(ctx)
    e = lambda k: torch.full((k,), 77, dtype=torch.int32, device="cuda")  # noqa: E731
    t = i(table).view(n, -1)
    outs = [t, e(n), e(n), e(1), e(n + 1), e(n_slots), e(n_slots)]
    gdn.gdn_kv_plan(i(ctx), i(new), i(owned), i(free), i([len(free) if n_free is None else n_free]), t, page, n_pages,
                    *outs[1:])
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in outs]


def plan_inputs(seed, n, page, ctx_max, new_max, spare=0):
    r = np.random.default_rng(seed)
    ctx = r.integers(0, ctx_max + 1, n)
    new = np.where(r.random(n) < 0.2, 0, r.integers(0, new_max + 1, n))
    owned = -(-ctx // page) + np.where(r.random(n) < 0.2, r.integers(0, 3, n), 0)  # some pages ahead, as after a rollback
    need = np.maximum(owned, -(-(ctx + new) // page))
    width = int(need.max()) + 2
    n_pages = int(need.sum()) + 10
    order = r.permutation(n_pages)
    table = np.full((n, width), -1)
    at = 0
    for s in range(n):
        table[s, : owned[s]] = order[at: at + owned[s]]
        at += owned[s]
    return ctx.tolist(), new.tolist(), owned.tolist(), order[at:].tolist(), table.tolist(), width, n_pages


@pytest.mark.parametrize("n,page,ctx_max,new_max", [(1, 16, 0, 1), (1, 1, 50, 40), (3, 16, 100, 1), (64, 24, 900, 1),
                                                   (300, 8, 50, 30), (1024, 16, 300, 2), (2500, 7, 40, 9),
                                                   (40, 64, 4000, 3000)])
def test_plan(torch, n, page, ctx_max, new_max):
    ctx, new, owned, free, table, width, n_pages = plan_inputs(n + page, n, page, ctx_max, new_max)
    n_slots = sum(new) + 5
    *want, short = plan_reference(ctx, new, owned, free, table, page, width, n_slots)
    assert not short
    assert plan_call(torch, ctx, new, owned, free, table, page, n_pages, n_slots) == want


def test_plan_without_tokens(torch):
    ctx, new, owned, free, table, width, n_pages = plan_inputs(5, 20, 16, 100, 0)
    *want, _ = plan_reference(ctx, new, owned, free, table, 16, width, 0)
    assert plan_call(torch, ctx, new, owned, free, table, 16, n_pages, 0) == want
    *want, _ = plan_reference(ctx, new, owned, [], table, 16, width, 3)
    assert plan_call(torch, ctx, new, owned, [], table, 16, n_pages, 3) == want


@pytest.mark.parametrize("cut", [0, 1, 7, 40])
def test_plan_out_of_pages(torch, cut):
    from serving_gdn_decode_gb300 import _native as nat
    ctx, new, owned, free, table, width, n_pages = plan_inputs(11, 1500, 8, 60, 20)
    free = free[:cut]
    n_slots = sum(new)
    *want, short = plan_reference(ctx, new, owned, free, table, 8, width, n_slots)
    assert short
    assert plan_call(torch, ctx, new, owned, free, table, 8, n_pages, n_slots) == want
    assert status() == nat.GDN_DEVICE_OUT_OF_PAGES


def test_plan_bad_requests(torch):
    """Impossible numbers are not served; the requests around them are."""
    from serving_gdn_decode_gb300 import _native as nat
    page, width = 8, 4
    ctx = [5, -1, 8, 30, 8, 3, 2 ** 31 - 1]
    new = [5, 1, -3, 1, 100, 1, 2 ** 31 - 1]
    owned = [1, 0, 1, 2, 1, 1, 9]
    table = [[10, -1, -1, -1], [-1] * 4, [11, -1, -1, -1], [12, 13, -1, -1], [14, -1, -1, -1], [15, -1, -1, -1], [-1] * 4]
    got = plan_call(torch, ctx, new, owned, [3, 2, 1], table, page, 20, 110)
    assert status() == nat.GDN_DEVICE_BAD_REQUEST
    t, kv, own, left, start, slots, pos = got
    assert kv == [10, 0, 0, 0, 8, 4, 0] and own == [2, 0, 1, 2, 1, 1, 9] and left == [2]
    assert t[0] == [10, 1, -1, -1] and t[1:] == table[1:]
    assert start[:7] == [0, 5, 6, 6, 7, 107, 108]
    assert slots[:5] == [85, 86, 87, 8, 9] and slots[5:107] == [-1] * 102 and slots[107] == 15 * 8 + 3
    assert pos[:5] == [5, 6, 7, 8, 9] and pos[107] == 3
    # fewer slots than tokens: the first ones are written
    got = plan_call(torch, [0], [6], [0], [1], [[-1]], 8, 4, 4)
    assert got[5] == [8, 9, 10, 11] and status() == nat.GDN_DEVICE_BAD_REQUEST
    # a stack size past the array
    got = plan_call(torch, [0], [6], [0], [1], [[-1]], 8, 4, 6, n_free=5)
    assert got[3] == [0] and got[5] == [8, 9, 10, 11, 12, 13] and status() == nat.GDN_DEVICE_BAD_REQUEST
    # page numbers that the cache does not have give no slot
    got = plan_call(torch, [0], [6], [0], [4], [[-1]], 8, 4, 6)
    assert got[5] == [-1] * 6 and status() == nat.GDN_DEVICE_BAD_PAGE


# ------------------------------------------------------------------ together


def test_steps_together(torch):
    """Six steps of ragged windows with a rollback, plan to attention, against attention over plainly
    kept keys and values."""
    import serving_gdn_decode_gb300 as gdn
    n_seqs, n_q, n_kv, dim, page, width = 3, 4, 2, 64, 4, 12
    g = torch.Generator().manual_seed(4)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    n_pages = 30
    kc, vc = (torch.full((n_pages, n_kv, page, dim), math.nan, device="cuda") for _ in range(2))
    table = torch.full((n_seqs, width), -1, dtype=torch.int32, device="cuda")
    state = [i32([0] * n_seqs), i32([0] * n_seqs), i32([n_pages])]  # lengths, owned, free
    free = torch.randperm(n_pages, generator=g).to(torch.int32).cuda()
    cs = table_of(torch, 64, dim)
    axes = [0] * (dim // 2)
    keys, values = [[] for _ in range(n_seqs)], [[] for _ in range(n_seqs)]
    for step, new in enumerate([[5, 1, 9], [1, 1, 1], [4, 4, 4], [1, 0, 1], [2, 3, 1], [1, 1, 1]]):
        n = sum(new)
        outs = [torch.empty(k, dtype=torch.int32, device="cuda") for k in (n_seqs, n_seqs, 1, n_seqs + 1, n, n)]
        gdn.gdn_kv_plan(state[0], i32(new), state[1], free, state[2], table, page, n_pages, *outs)
        kv, owned, left, start, slots, pos = outs
        q, k, v = (torch.randn(n, h, dim, generator=g) for h in (n_q, n_kv, n_kv))
        qd = q.cuda()
        gdn.gdn_rope_store(qd, k.cuda(), v.cuda(), pos, cs.cuda(), slots, kc, vc, qd)
        out = torch.empty_like(qd)
        ws = torch.empty(gdn.gdn_attn_workspace_size(qd, kc, n_seqs), dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_paged(qd, kc, vc, table, kv, start, out, ws)
        ref, row = torch.zeros(n, n_q, dim, dtype=torch.float64), 0
        for s in range(n_seqs):
            for t in range(new[s]):
                at = torch.tensor([[len(keys[s])]])
                rot = lambda x: rope_reference(torch, x, at, cs, axes, False)[0]  # noqa: E731
                keys[s].append(rot(k[row: row + 1]))
                values[s].append(v[row].double())
                kk, vv = torch.stack(keys[s], 1), torch.stack(values[s], 1)
                qq = rot(q[row: row + 1]).view(n_kv, n_q // n_kv, dim)
                p = torch.softmax(torch.einsum("hgd,hkd->hgk", qq, kk) / math.sqrt(dim), -1)
                ref[row] = torch.einsum("hgk,hkd->hgd", p, vv).reshape(n_q, dim)
                row += 1
        assert rel(out, ref) <= TOL["f32"]
        if step == 2:  # two of the four drafted tokens are rejected
            kv = kv - 2
            keys, values = [x[:-2] for x in keys], [x[:-2] for x in values]
        assert kv.tolist() == [len(x) for x in keys]
        state = [kv, owned, left]
    assert int(state[2]) == n_pages - sum(state[1].tolist())


def test_hybrid_example(torch, capsys):
    """The example's decode steps (captured and replayed) end where one pass over all tokens does.  Both
    paths are f32; eight layers of sums of 512 to 1024 terms, each step's rounding amplified by the
    normalisations: 1e-3 of the logits is a hundred times what f32 leaves and far below any slip."""
    from serving_gdn_decode_gb300 import hybrid_step
    assert hybrid_step.main(["--requests", "5", "--prompt", "37", "--steps", "20", "--check"]) <= 1e-3
    assert "device status 0" in capsys.readouterr().out


def test_calls_on_two_streams(torch):
    """Calls that overlap on two streams, each with its own workspace, and calls back to back on one stream
    that share one, give what they give alone."""
    import serving_gdn_decode_gb300 as gdn
    cases = [Case(torch, "bf16", [3000 + 500 * i, 700, 64], dim=128, group=4, seed=i) for i in range(4)]
    alone = [c.run(torch).clone() for c in cases]
    for c in cases:
        c.out.fill_(9.0)
    size = max(gdn.gdn_attn_workspace_size(c.q_dev, c.k_dev, 3) for c in cases)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate(cases):
            gdn.gdn_attn_paged(c.q_dev, c.k_dev, c.v_dev, c.table, c.kv_lens, c.start, c.out, work[i % 2],
                               stream=streams[i % 2])
    torch.cuda.synchronize()
    for c, want in zip(cases, alone):
        assert torch.equal(c.out, want)


def test_a_step_follows_what_is_before_it(torch):
    """Short kernels launched back to back read what the ones before them wrote: a chain of in-place
    rotations by one position each, mixed with torch's kernels, ends at the sum of them."""
    import serving_gdn_decode_gb300 as gdn
    n, steps = 8, 200
    table = table_of(torch, 2, 64).cuda()
    pos = torch.ones(n, dtype=torch.int32, device="cuda")
    q = torch.randn(n, 2, 64, generator=torch.Generator().manual_seed(0)).cuda()
    k = q.clone()
    start = q.double().cpu()
    for i in range(steps):
        gdn.gdn_rope(q, k, pos, table, q, k)
        if i % 3 == 0:
            q.mul_(2.0)
            q.mul_(0.5)
    angle = steps * 10000.0 ** (-torch.arange(32, dtype=torch.float64) * 2 / 64)
    a, b = start[..., :32], start[..., 32:]
    want = torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)
    # each step is off by 2^-24 in its cosines and 2^-23 in its sums: 200 steps of either sign
    assert rel(q, want) <= 200 * 3 * 2.0 ** -24 and torch.equal(q, k)
