"""GPU tests of the 8-bit paged cache (gdn_kv_store_fp8, gdn_kv_load_fp8,
gdn_attn_paged_fp8) against plain implementations in 64 bits.

Tolerances, from the arithmetic:
* store: scales are powers of two, so x / scale and code * (old / scale) are exact
  in f32 and a code is the one rounding of it: codes and scales are equal.
* load: code * scale is exact in f32 and bf16 for those scales: equal; for scales
  of any value one rounding of f32 (2^-24 of the value), with bf16's 2^-8 after it.
* f32 attention: q is hi + lo in f16, 2^-22 of it, and codes are exact: a product is
  off by 2^-22 of |q||k| at most.  With sum |q k| * scale below 24 for these inputs a
  score is off by 6e-6, a probability, hi + lo again, and the output by at most twice
  that and 2^-22: 2e-5 with room for the sums in f32.
* bf16 attention: q is exact; a probability has f16's rounding, 2^-11 of it at most
  and of either sign, 2^-12 root-mean-square or less; then the result's one rounding,
  2^-8 of an element at most, 2^-9 root-mean-square or less: rel-L2 2^-9 + 2^-12 + 2e-5.
"""
import math

import numpy as np
import pytest

from test_gpu_paged import clean_status, rel, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu

TOL = {"f32": 2e-5, "bf16": 2.0 ** -9 + 2.0 ** -12 + 2e-5}
TOP = 448.0


def dtype_of(torch, name):  # noqa: F811
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def nearest(torch, y):  # noqa: F811
    """y (64 bits) on e4m3's grid, ties to even; what is not finite is NaN."""
    fine = y.isfinite()
    z = torch.where(fine, y, 0.0)
    e = torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6)))
    step = 2.0 ** (e - 3)
    z = (torch.round(z / step) * step).clamp(-TOP, TOP)
    return torch.where(fine, z, math.nan)


def least_scale(top):
    e = -110
    while e < 119 and top > TOP * 2.0 ** e:
        e += 1
    return 2.0 ** e


def same(torch, got, ref):  # noqa: F811
    got, ref = got.double().cpu(), ref.double().cpu()
    assert got.shape == ref.shape
    bad = ~((got == ref) | (got.isnan() & ref.isnan()))
    assert not bad.any(), (bad.nonzero()[:5].tolist(), got[bad][:5].tolist(), ref[bad][:5].tolist())


# ------------------------------------------------------------------ store and load


class Store:
    """An 8-bit cache with something in it, and a step's k and v to store."""

    def __init__(self, torch, dtype, slots, n_pages=8, n_kv=2, page=16, dim=64, layout="hnd", seed=0, wide=True, values=None):  # noqa: F811
        g = torch.Generator().manual_seed(seed)
        self.torch, self.page, self.n_kv, self.dim, self.slots = torch, page, n_kv, dim, list(slots)
        n = len(self.slots)
        pad = 0 if wide else 1  # rows that are aligned to an element only
        fused = torch.zeros(max(n, 1), 2 * n_kv * dim + pad, dtype=dtype_of(torch, dtype), device="cuda")
        x = torch.randn(2, n, n_kv, dim, generator=g) * torch.exp2(torch.randint(-6, 6, (2, n, n_kv, 1), generator=g).float())
        if values is not None:
            values(x)
        fused[:n, pad:] = x.permute(1, 0, 2, 3).reshape(n, 2 * n_kv * dim).to(fused)
        self.k, self.v = (t.unflatten(1, (n_kv, dim)) for t in fused[:n, pad:].split(n_kv * dim, 1))
        self.cache, self.scale = [], []
        both = torch.zeros(n_pages, 2, n_kv, page, dim, dtype=torch.uint8, device="cuda")
        for i in range(2):
            codes = (torch.randn(n_pages, n_kv, page, dim, generator=g) * 60).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            if layout == "nhd":
                codes = codes.transpose(1, 2).contiguous().transpose(1, 2)
            elif layout == "both":
                both[:, i] = codes
                codes = both[:, i]
            self.cache.append(codes.view(torch.float8_e4m3fn))
            self.scale.append(torch.exp2(torch.randint(-9, 3, (n_pages, n_kv), generator=g).float()).cuda())

    def reference(self):
        torch, page = self.torch, self.page  # noqa: F811
        cache, scale = [c.double().cpu() for c in self.cache], [s.double().cpu() for s in self.scale]
        n_pages = cache[0].shape[0]
        i = 0
        while i < len(self.slots):
            j = i + 1
            while j < len(self.slots) and self.slots[i] >= 0 and self.slots[j] == self.slots[j - 1] + 1 and self.slots[j] % page:
                j += 1
            p, a = divmod(self.slots[i], page)
            out_of_order = i and self.slots[i - 1] >= 0 and self.slots[i - 1] // page == p
            if self.slots[i] >= 0 and p < n_pages and not out_of_order:
                for c, s, x in zip(cache, scale, (self.k, self.v)):
                    for h in range(self.n_kv):
                        rows = x[i:j, h].double().cpu()
                        new = least_scale(float(torch.where(rows.isfinite(), rows.abs(), 0.0).max()))
                        old = float(s[p, h])
                        if a and math.isfinite(old):
                            new = max(new, old)
                        if a and new != old:
                            by = old / new if math.isfinite(old) and old >= 0 else math.nan
                            c[p, h, :a] = nearest(torch, c[p, h, :a] * by)
                        c[p, h, a : a + j - i] = nearest(torch, rows / new)
                        s[p, h] = new
            i = j
        return cache, scale

    def call(self, stream=None):
        import serving_gdn_decode_gb300 as gdn
        slots = self.torch.tensor(self.slots, dtype=self.torch.int32, device="cuda")
        gdn.gdn_kv_store_fp8(self.k, self.v, slots, *self.cache, *self.scale, stream=stream)
        self.torch.cuda.synchronize()

    def check(self):
        cache, scale = self.reference()
        self.call()
        for got, ref in zip(self.cache + self.scale, cache + scale):
            same(self.torch, got, ref)


def runs_of(page, n_pages, spec):
    """Slots of runs (page number, first place, tokens)."""
    return [p * page + a + i for p, a, n in spec for i in range(n)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("page", [1, 16, 24, 128])
def test_store_runs(torch, dtype, dim, page):  # noqa: F811
    """Whole pages, beginnings, middles and ends of pages, single tokens, idle tokens between."""
    cut = lambda n: max(1, min(n, page))  # noqa: E731
    spec = [(3, 0, page), (1, 0, cut(5)), (6, page // 2, page - page // 2), (0, page - 1, 1), (5, cut(2) - 1, 1)]
    slots = runs_of(page, 8, spec)
    Store(torch, dtype, slots, page=page, dim=dim, n_kv=3).check()
    Store(torch, dtype, [-1] + slots[:page] + [-1, -1] + slots[page:] + [-1], page=page, dim=dim, n_kv=1, seed=1).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
@pytest.mark.parametrize("wide", [True, False])
def test_store_layouts(torch, dtype, layout, wide):  # noqa: F811
    spec = [(2, 3, 13), (0, 0, 16), (7, 0, 9), (4, 15, 1)]
    Store(torch, dtype, runs_of(16, 8, spec), dim=96, n_kv=2, layout=layout, wide=wide).check()


@pytest.mark.parametrize("dtype,page,dim,n_kv", [("bf16", 16, 128, 8), ("bf16", 64, 128, 8), ("f32", 200, 256, 1), ("bf16", 1, 64, 4), ("f32", 33, 64, 3)])
def test_store_long_runs(torch, dtype, page, dim, n_kv):  # noqa: F811
    """Prompts of thousands of tokens over shuffled pages, beginning inside one."""
    n_pages = 4200 // page + 4
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(3)).tolist()
    first = page // 3
    slots = [order[i // page] * page + i % page for i in range(first, first + 3000)]
    s = Store(torch, dtype, slots, n_pages=n_pages, page=page, dim=dim, n_kv=n_kv, seed=4)
    before = [c.view(torch.uint8).clone() for c in s.cache]
    x = [t.double() for t in (s.k, s.v)]
    s.call()
    # page by page against the values themselves: each is within half a step of its code
    at = torch.tensor(slots, device="cuda")
    for c, sc, y, old in zip(s.cache, s.scale, x, before):
        got = c[at // page, :, at % page].double()
        scale = sc[at // page].double()[:, :, None]
        ref = nearest(torch, (y / scale).cpu()).cuda()
        same(torch, got, ref)
        for p in set((at // page).tolist()):
            rows = (at // page == p).nonzero()[:, 0]
            tops = y[rows].abs().amax((0, 2)).tolist()
            begins = int(at[rows[0]]) % page == 0
            for h, top in enumerate(tops):
                assert float(sc[p, h]) == least_scale(top) or (not begins and float(sc[p, h]) >= least_scale(top))
        untouched = torch.ones(c.shape[0], c.shape[2], dtype=torch.bool, device="cuda")
        untouched[at // page, at % page] = False
        untouched[slots[0] // page] = False  # its earlier codes may have been rounded again
        now = c.view(torch.uint8).transpose(1, 2)
        assert torch.equal(now[untouched], old.transpose(1, 2)[untouched])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_store_special_values(torch, dtype):  # noqa: F811
    """NaN and infinities, zeros, borders of a scale, the largest and smallest values."""
    big, least = (3.3895313892515355e38, 2.0 ** -126) if dtype == "bf16" else (3.4028234663852886e38, 2.0 ** -149)

    def values(x):
        x[0, 0, 0, :4] = x.new_tensor([math.nan, math.inf, -math.inf, -0.0])
        x[0, 1] = 0.0
        x[1, 0] = math.nan
        x[1, 1, 0] = 0.0
        x[1, 1, 0, 0] = 448.0  # on the border: scale 1
        x[1, 1, 1] = 0.0
        x[1, 1, 1, 0] = 450.0 if dtype == "bf16" else 448.00003
        x[0, 2, 0, 1] = big
        x[0, 2, 1] = least
        x[1, 2, 0] = 2.0 ** -110
        x[1, 2, 1] = x[1, 2, 1] * 0 + 2.0 ** -101 * 1.75

    # a page each, then one page that they share
    Store(torch, dtype, [0, 16, 32], dim=32, values=values).check()
    Store(torch, dtype, [48, 49, 50], dim=32, values=values).check()
    Store(torch, dtype, [53, 54, 55], dim=32, values=values).check()


@pytest.mark.parametrize("dim,page", [(64, 16), (256, 40)])
def test_store_grows_and_keeps(torch, dim, page):  # noqa: F811
    """Token by token: the scale grows when a token needs it, codes before are rounded again, never shrinks."""
    import serving_gdn_decode_gb300 as gdn
    s = Store(torch, "f32", [0], dim=dim, page=page, n_kv=2, n_pages=2)
    cache, scale = [c.double().cpu() for c in s.cache], [x.double().cpu() for x in s.scale]
    g = torch.Generator().manual_seed(5)
    for i in range(page):
        size = 2.0 ** [0, 3, -2, 3, 10, 1, 30, -30, 31][i % 9]
        k, v = (size * torch.randn(2, 1, 2, dim, generator=g)).cuda()
        gdn.gdn_kv_store_fp8(k, v, torch.tensor([page + i], dtype=torch.int32, device="cuda"), *s.cache, *s.scale)
        for c, sc, x in zip(cache, scale, (k, v)):
            for h in range(2):
                row, old = x[0, h].double().cpu(), float(sc[1, h])
                new = max(least_scale(float(row.abs().max())), old if i else 0.0)
                c[1, h, :i] = nearest(torch, c[1, h, :i] * (old / new))
                c[1, h, i] = nearest(torch, row / new)
                sc[1, h] = new
    torch.cuda.synchronize()
    for got, ref in zip(s.cache + s.scale, cache + scale):
        same(torch, got, ref)


def test_store_old_scales_that_are_none(torch):  # noqa: F811
    """0: the codes before become zero; negative, infinite, NaN: NaN; another positive value is taken as it is."""
    for old in (0.0, -1.0, math.inf, math.nan):
        s = Store(torch, "bf16", [5, 6])
        for x in s.scale:
            x[0] = old
        s.check()
    s = Store(torch, "f32", [5, 6])
    for x in s.scale:
        x[0] = 1e9
    k, v, old = s.k.double(), s.v.double(), [c[0].view(torch.uint8).clone() for c in s.cache]
    s.call()
    for c, x, y, o in zip(s.cache, s.scale, (k, v), old):
        assert bool((x[0] == 1e9).all())
        assert torch.equal(c[0, :, :5].view(torch.uint8), o[:, :5])  # not touched
        got = c[0, :, 5:7].double().transpose(0, 1) * 1e9
        assert bool(((got - y).abs() <= y.abs() * (2.0 ** -4 + 2.0 ** -22) + 1e9 * 2.0 ** -10).all())


def test_store_bad_slots_are_reported(torch):  # noqa: F811
    from serving_gdn_decode_gb300 import _native as nat
    Store(torch, "bf16", [3, 8 * 16, 8 * 16 + 1, 20, -7]).check()
    assert status() == nat.GDN_DEVICE_BAD_PAGE
    Store(torch, "bf16", [(1 << 31) - 1, 0]).check()
    assert status() == nat.GDN_DEVICE_BAD_PAGE
    Store(torch, "bf16", [19, 18, 20, 0, 1]).check()  # slots of one page out of order: the first run of them is stored
    assert status() == nat.GDN_DEVICE_BAD_REQUEST
    Store(torch, "f32", [3, 3]).check()
    assert status() == nat.GDN_DEVICE_BAD_REQUEST


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page,layout", [(16, 1, "hnd"), (64, 16, "nhd"), (80, 24, "both"), (128, 16, "hnd"), (256, 33, "hnd")])
@pytest.mark.parametrize("wide", [True, False])
def test_load(torch, dtype, dim, page, layout, wide):  # noqa: F811
    import serving_gdn_decode_gb300 as gdn
    n_pages = 9
    g = torch.Generator().manual_seed(6)
    slots = torch.randperm(n_pages * page, generator=g)[: max(1, 3 * page)].to(torch.int32)
    slots = torch.cat([slots, slots[:1], torch.tensor([-1, -5], dtype=torch.int32)]).cuda()
    s = Store(torch, dtype, range(len(slots)), n_pages=n_pages, page=page, dim=dim, n_kv=3, layout=layout, wide=wide)
    s.cache[0].view(torch.uint8)[1, 0, 0, 0] = 0x7F  # a NaN
    ref = []
    for c, sc, x in zip(s.cache, s.scale, (s.k, s.v)):
        at = slots.clamp(min=0).long()
        y = c[at // page, :, at % page].double() * sc[at // page].double()[:, :, None]
        ref.append(torch.where((slots >= 0)[:, None, None], y, x.double()))
    gdn.gdn_kv_load_fp8(slots, *s.cache, *s.scale, s.k, s.v)
    torch.cuda.synchronize()
    for got, want in zip((s.k, s.v), ref):
        same(torch, got, want)


def test_load_any_scale_and_bad_slots(torch):  # noqa: F811
    import serving_gdn_decode_gb300 as gdn
    from serving_gdn_decode_gb300 import _native as nat
    for dtype, eps in (("f32", 2.0 ** -24), ("bf16", 2.0 ** -8 + 2.0 ** -23)):
        s = Store(torch, dtype, range(32), seed=7)
        for x in s.scale:
            x.copy_(torch.rand(x.shape, generator=torch.Generator().manual_seed(8)) + 0.01)
        slots = torch.arange(40, 72, dtype=torch.int32, device="cuda")
        gdn.gdn_kv_load_fp8(slots, *s.cache, *s.scale, s.k, s.v)
        for c, sc, got in zip(s.cache, s.scale, (s.k, s.v)):
            ref = c[slots.long() // 16, :, slots.long() % 16].double() * sc[slots.long() // 16].double()[:, :, None]
            assert bool(((got.double() - ref).abs() <= eps * ref.abs()).all())
        assert status() == 0
        slots[3] = 8 * 16
        keep = s.k.clone()
        gdn.gdn_kv_load_fp8(slots, *s.cache, *s.scale, s.k, s.v)
        torch.cuda.synchronize()
        assert status() == nat.GDN_DEVICE_BAD_PAGE
        assert bool(s.k[3].isnan().all()) and bool(s.v[3].isnan().all())
        others = torch.arange(32, device="cuda") != 3
        assert torch.equal(s.k[others], keep[others])


def test_store_and_load_no_tokens(torch):  # noqa: F811
    import serving_gdn_decode_gb300 as gdn
    s = Store(torch, "bf16", [])
    before = [c.view(torch.uint8).clone() for c in s.cache]
    s.call()
    gdn.gdn_kv_load_fp8(torch.zeros(0, dtype=torch.int32, device="cuda"), *s.cache, *s.scale, s.k, s.v)
    torch.cuda.synchronize()
    for c, b in zip(s.cache, before):
        assert torch.equal(c.view(torch.uint8), b)


# ------------------------------------------------------------------ attention


class Case:
    """An 8-bit paged cache with requests in it.  Slots that no request holds are NaN, as are the scales of
    pages that no request has."""

    def __init__(self, torch, dtype, lens, wins=None, n_kv=2, group=2, dim=128, page=16, layout="hnd", seed=0,  # noqa: F811
                 extra=3, max_pages=None, fused_q=False, spread=3):
        g = torch.Generator().manual_seed(seed)
        dt = dtype_of(torch, dtype)
        self.lens, self.wins = list(lens), list(wins) if wins is not None else [1] * len(lens)
        self.n_kv, self.group, self.dim, self.page = n_kv, group, dim, page
        pages = [-(-n // page) for n in self.lens]
        n_pages = sum(pages) + extra
        order = torch.randperm(n_pages, generator=g)
        width = max(max(pages), 1) if max_pages is None else max_pages
        table = torch.full((len(lens), width), -1, dtype=torch.int32)
        filled = torch.zeros(n_pages, page, dtype=torch.bool)
        used = torch.zeros(n_pages, dtype=torch.bool)
        at = 0
        for s, n in enumerate(self.lens):
            mine = order[at : at + pages[s]]
            table[s, : pages[s]] = mine.int()
            used[mine] = True
            rows = torch.zeros(pages[s] * page, dtype=torch.bool)
            rows[:n] = True
            filled[mine] = rows.view(pages[s], page)
            at += pages[s]
        self.cache, self.scale = [], []
        for _ in range(2):
            # codes of about 1 / scale: scales differ from page to page
            sc = torch.exp2(torch.randint(-spread, spread + 1, (n_pages, n_kv), generator=g).float()) / 64
            x = torch.randn(n_pages, n_kv, page, dim, generator=g) / sc[:, :, None, None]
            x = torch.where(filled[:, None, :, None], x.clamp(-TOP, TOP), math.nan)
            self.cache.append(x.to(torch.float8_e4m3fn).float())  # the codes' values
            self.scale.append(torch.where(used[:, None], sc, math.nan))
        n = sum(self.wins)
        self.q = (1.5 * torch.randn(n, n_kv * group, dim, generator=g)).to(dt)
        self.table = table.cuda()
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32).cuda()
        self.start = torch.tensor([0] + list(np.cumsum(self.wins)), dtype=torch.int32).cuda()
        dev = [self.codes(torch, i) for i in range(2)]
        if layout == "nhd":  # [page, slot, head, dim] in memory
            dev = [c.transpose(1, 2).contiguous().transpose(1, 2) for c in dev]
        elif layout == "both":  # K and V of a page side by side
            both = torch.stack(dev, 1).contiguous()
            dev = [both[:, 0], both[:, 1]]
        self.cache_dev = [c.view(torch.float8_e4m3fn) for c in dev]
        self.scale_dev = [s.cuda() for s in self.scale]
        self.q_dev = self.q.cuda()
        if fused_q:  # rows of a wider projection
            wide = torch.zeros(n, (n_kv * group + 2 * n_kv) * dim, dtype=dt, device="cuda")
            view = wide[:, : n_kv * group * dim].unflatten(1, (n_kv * group, dim))
            view.copy_(self.q_dev)
            self.q_dev = view
        self.out = torch.full((n, n_kv * group, dim), 7.0, dtype=dt, device="cuda")

    def codes(self, torch, i):  # noqa: F811
        return self.cache[i].to(torch.float8_e4m3fn).view(torch.uint8).cuda()

    def run(self, torch, scale=None, window=0, stream=None, start=True):  # noqa: F811
        import serving_gdn_decode_gb300 as gdn
        size = gdn.gdn_attn_fp8_workspace_size(self.q_dev, self.cache_dev[0], len(self.lens))
        # whatever the workspace holds must not matter
        ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        gdn.gdn_attn_paged_fp8(self.q_dev, *self.cache_dev, *self.scale_dev, self.table, self.kv_lens,
                               self.start if start else None, self.out, ws, scale=scale, window=window, stream=stream)
        torch.cuda.synchronize()
        return self.out

    def values(self, i, pages):
        return (self.cache[i][pages].double() * self.scale[i][pages].double()[:, :, None, None]).permute(1, 0, 2, 3) \
            .reshape(self.n_kv, -1, self.dim)

    def reference(self, torch, scale=None, window=0):  # noqa: F811
        scale = 1.0 / math.sqrt(self.dim) if scale is None else scale
        out = torch.zeros(self.q.shape, dtype=torch.float64)
        row = 0
        for s, (n, w) in enumerate(zip(self.lens, self.wins)):
            pages = self.table[s, : -(-n // self.page)].long().cpu().clamp(min=0)
            k, v = self.values(0, pages), self.values(1, pages)
            for t in range(w):
                hi = n - w + t + 1
                lo = max(0, hi - window) if window else 0
                if hi > 0:
                    q = self.q[row].double().view(self.n_kv, self.group, self.dim)
                    p = torch.softmax(scale * torch.einsum("hgd,hkd->hgk", q, k[:, lo:hi]), -1)
                    out[row] = torch.einsum("hgk,hkd->hgd", p, v[:, lo:hi]).reshape(-1, self.dim)
                row += 1
        return out

    def check(self, torch, dtype, **kw):  # noqa: F811
        ref = self.reference(torch, **{k: v for k, v in kw.items() if k in ("scale", "window")})
        got = self.run(torch, **kw)
        assert rel(got, ref) <= TOL[dtype]
        # row by row, none far from its values
        got64, worst = got.double().cpu(), 0.0
        for r in range(len(ref)):
            if float(ref[r].norm()):
                worst = max(worst, float((got64[r] - ref[r]).norm() / ref[r].norm()))
        assert worst <= 3 * TOL[dtype], worst
        # rows without a key are exactly zero
        empty = (ref == 0).all(-1).all(-1)
        assert not got[empty.to(got.device)].any()


EDGES = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 129, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 8])
def test_attn_lengths(torch, dtype, dim, group):  # noqa: F811
    Case(torch, dtype, EDGES, dim=dim, group=group, n_kv=2).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [9, 16, 17, 40, 70])
def test_attn_large_groups(torch, dtype, dim, group):  # noqa: F811
    """More query heads per key head than one row tile takes, up to several row blocks."""
    Case(torch, dtype, [200, 1, 77], dim=dim, group=group, n_kv=1).check(torch, dtype)
    Case(torch, dtype, [70, 500, 5], dim=dim, group=group, n_kv=2, page=24).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 3, 8, 24, 32, 48, 64, 200])
@pytest.mark.parametrize("layout", ["hnd", "nhd", "both"])
def test_attn_pages_and_layouts(torch, dtype, dim, page, layout):  # noqa: F811
    Case(torch, dtype, [37, 200, 1, 401], page=page, layout=layout, dim=dim, group=4, n_kv=3, fused_q=True).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 2), (128, 5), (256, 8)])
@pytest.mark.parametrize("page", [16, 24])
def test_attn_windows_of_tokens(torch, dtype, dim, group, page):  # noqa: F811
    """Ragged windows; more tokens than keys (the first rows see none); idle requests."""
    c = Case(torch, dtype, [100, 3, 40, 0, 64, 7], wins=[4, 5, 1, 0, 7, 7], dim=dim, group=group, page=page)
    c.check(torch, dtype)
    c.check(torch, dtype, window=33)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [1, 5, 16, 64, 100, 1 << 30, (1 << 32) - 1])
@pytest.mark.parametrize("page", [16, 24])
def test_attn_sliding_window(torch, dtype, window, page):  # noqa: F811
    Case(torch, dtype, [300, 64, 65, 5, 1], wins=[1, 3, 1, 2, 1], page=page).check(torch, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 4), (128, 9), (256, 4), (256, 14)])
@pytest.mark.parametrize("page", [16, 24, 32])
def test_attn_unseen_codes_and_scales(torch, dtype, dim, group, page):  # noqa: F811
    """NaN in what a row does not see: keys behind its window or after its token, whole pages behind the window
    and their scales, table entries that are gone."""
    c = Case(torch, dtype, [150, 90, 33], wins=[3, 4, 2], dim=dim, group=group, page=page, n_kv=1)
    window = 40
    ref = c.reference(torch, window=window)
    for s, (n, w) in enumerate(zip(c.lens, c.wins)):
        first = max(0, n - w + 1 - window)  # the first key that any row sees
        for j in range(first // page):
            p = int(c.table[s, j])
            for x in c.cache_dev:
                x.view(torch.uint8)[p] = 0x7F
            for x in c.scale_dev:
                x[p] = math.nan if j % 2 else math.inf
            if j % 3 == 0:
                c.table[s, j] = -1 if j % 2 else 1 << 30
        for key in range(first // page * page, first):
            for x in c.cache_dev:
                x.view(torch.uint8)[int(c.table[s, key // page]), :, key % page] = 0xFF
    got = c.run(torch, window=window)
    assert rel(got, ref) <= TOL[dtype]
    # the last key is NaN: only the rows of the last token see it
    c = Case(torch, dtype, [70, 33], wins=[3, 2], dim=dim, group=group, page=page, n_kv=1)
    ref = c.reference(torch)
    for s, n in enumerate(c.lens):
        for x in c.cache_dev:
            x.view(torch.uint8)[int(c.table[s, (n - 1) // page]), :, (n - 1) % page] = 0x7F
    got = c.run(torch)
    last = torch.zeros(len(got), dtype=torch.bool, device="cuda")
    last[c.start[1:].long() - 1] = True
    assert bool(got[last].isnan().all())
    assert rel(got[~last], ref[~last.cpu()]) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_scores_of_minus_infinity(torch, dtype):  # noqa: F811
    """q with an infinity: scores are infinite, the result is NaN, and no other row's is."""
    c = Case(torch, dtype, [100, 40, 300], group=4)
    ref = c.reference(torch)
    c.q_dev[1, 2, 5] = -math.inf
    c.q_dev[2, 0, 0] = math.nan
    got = c.run(torch)
    mask = torch.zeros(3, 8, dtype=torch.bool)
    mask[1, 2] = mask[2, 0] = True
    assert bool(got.cpu()[mask].isnan().all())
    assert rel(got.cpu()[~mask], ref[~mask]) <= TOL[dtype]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 8), (128, 4), (256, 2)])
def test_attn_long_and_split(torch, dtype, dim, group):  # noqa: F811
    Case(torch, dtype, [30011, 5000], n_kv=1, group=group, dim=dim).check(torch, dtype)
    Case(torch, dtype, [9001], wins=[3], n_kv=1, group=group, dim=dim, page=24).check(torch, dtype)


def test_attn_many_requests(torch):  # noqa: F811
    r = np.random.RandomState(4)
    Case(torch, "bf16", r.randint(0, 90, 700).tolist(), n_kv=1, group=2, dim=64).check(torch, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("max_pages", [8, 16, 17, 100])
def test_attn_table_width(torch, dtype, max_pages):  # noqa: F811
    """Tables that bound the keys to a few tiles, and wider ones over the same requests."""
    Case(torch, dtype, [128, 1, 77, 0, 128], max_pages=max_pages).check(torch, dtype)


@pytest.mark.parametrize("scale", [0.0, -0.3, 2.0])
def test_attn_scales(torch, scale):  # noqa: F811
    Case(torch, "f32", [100, 40], spread=1).check(torch, "f32", scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [8, 16, 24, 64])
def test_attn_scales_far_apart(torch, dtype, page):  # noqa: F811
    """Pages whose value scales differ by up to 2^200 with the largest not weighted at all, and large and small key
    scales and queries."""
    c = Case(torch, dtype, [160, 70, 200], page=page, group=3, n_kv=1, spread=0)
    r = np.random.RandomState(1)
    for s in range(3):
        for j in range(-(-c.lens[s] // page)):
            p = int(c.table[s, j])
            by = 2.0 ** int(r.randint(-100, 0)) if j % 3 else 1.0
            c.scale[1][p] *= by
            if j % 3 == 2:  # keys far below the others: their probabilities are zero, their values huge
                c.cache[0][p] = torch.where(c.cache[0][p].isnan(), c.cache[0][p], -448.0)
                c.scale[0][p] = 2.0 ** 6
                c.scale[1][p] = 2.0 ** 100
    c.q = c.q.abs()  # against keys of -448 * 64 every score is far below
    for i in range(2):
        c.cache_dev[i].view(torch.uint8).copy_(c.codes(torch, i))
        c.scale_dev[i].copy_(c.scale[i])
    c.q_dev.copy_(c.q)
    c.check(torch, dtype)
    for by in (2.0 ** 60, 2.0 ** -60):  # q and the key scales against one another: the scores stay
        c.q_dev.copy_((c.q.double() * by).to(c.q.dtype))
        c.scale_dev[0].copy_((c.scale[0].double() / by).float())
        assert rel(c.run(torch), c.reference(torch)) <= TOL[dtype]


def test_attn_q_of_wide_range(torch):  # noqa: F811
    """q rows whose elements differ by up to 2^30, and rows of zeros."""
    for dtype in ("bf16", "f32"):
        c = Case(torch, dtype, [100, 64], group=4, spread=0)
        g = torch.Generator().manual_seed(3)
        q = c.q.float() * torch.exp2(-torch.randint(0, 31, c.q.shape, generator=g).float())
        q[0, 1] = 0.0
        c.q = q.to(c.q.dtype)
        c.q_dev.copy_(c.q)
        c.check(torch, dtype)


def test_attn_small_probabilities_add_up(torch):  # noqa: F811
    """One key far above 60000 others that together weigh as much: what a probability loses below f16's range must not
    be seen."""
    n, page = 60001, 64
    c = Case(torch, "bf16", [n], n_kv=1, group=1, dim=64, page=page, spread=0)
    c.q.zero_()
    c.q[0, 0, 0] = 8.0  # at the default scale of 1/8 the score is element 0 of the key
    first = int(c.table[0, 0])
    c.cache[0][..., 0] *= 0.0  # scores of 0, and NaN where there is no key
    c.cache[0][first, 0, 0, 0] = TOP
    c.scale[0] *= 11.0 / TOP / c.scale[0]  # and one of 11: e^11 = 59874
    c.cache[1] = (c.cache[1] + 64.0).to(torch.float8_e4m3fn).float()  # values of mean 1, so that a lost tail shows
    for i in range(2):
        c.cache_dev[i].view(torch.uint8).copy_(c.codes(torch, i))
        c.scale_dev[i].copy_(c.scale[i])
    c.q_dev.copy_(c.q)
    c.check(torch, "bf16")


def test_attn_strided_q_other_stream_and_runs(torch):  # noqa: F811
    c = Case(torch, "bf16", [500, 33, 900], group=4, fused_q=True)
    a = c.run(torch).clone()
    stream = torch.cuda.Stream()
    for _ in range(3):
        c.out.fill_(3.0)
        torch.cuda.synchronize()
        assert torch.equal(c.run(torch, stream=stream), a)
    assert rel(a, c.reference(torch)) <= TOL["bf16"]
    assert torch.equal(c.run(torch, start=False), a)


def test_attn_writes_its_rows_only(torch):  # noqa: F811
    """Rows of q behind the last request, and columns beside the output, stay as they were."""
    import serving_gdn_decode_gb300 as gdn
    c = Case(torch, "bf16", [100, 30], group=2)
    ref = c.reference(torch)
    q = torch.cat([c.q_dev, c.q_dev, c.q_dev])
    wide = torch.full((6, 4 * 128 + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, 8 : 8 + 512].unflatten(1, (4, 128))
    ws = torch.empty(gdn.gdn_attn_fp8_workspace_size(q, c.cache_dev[0], 2), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_paged_fp8(q, *c.cache_dev, *c.scale_dev, c.table, c.kv_lens, c.start, out, ws)
    torch.cuda.synchronize()
    assert rel(out[:2], ref) <= TOL["bf16"]
    assert bool((wide[2:] == 5).all()) and bool((wide[:, :8] == 5).all()) and bool((wide[:, 520:] == 5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_output_aligned_to_an_element_only(torch, dtype):  # noqa: F811
    c = Case(torch, dtype, [100, 30, 700], group=2)
    a = c.run(torch).clone()
    wide = torch.zeros(3, 4 * 128 + 1, dtype=a.dtype, device="cuda")
    c.out = wide[:, 1:].unflatten(1, (4, 128))
    assert torch.equal(c.run(torch), a)


def test_attn_bad_data_is_reported(torch):  # noqa: F811
    from serving_gdn_decode_gb300 import _native as nat
    c = Case(torch, "bf16", [100, 30, 50])
    ref = c.reference(torch)
    good = c.table.clone()
    c.table[1, 1] = -1
    got = c.run(torch)
    assert status() == nat.GDN_DEVICE_BAD_PAGE
    assert bool(got[1].isnan().all()) and rel(got[[0, 2]], ref[[0, 2]]) <= TOL["bf16"]
    c.table.copy_(good)
    c.kv_lens[1] = -4
    got = c.run(torch)
    assert status() == nat.GDN_DEVICE_BAD_REQUEST
    assert not got[1].any() and rel(got[[0, 2]], ref[[0, 2]]) <= TOL["bf16"]
    c.kv_lens[1] = 30
    c.start[3] = 9
    got = c.run(torch)
    assert status() == nat.GDN_DEVICE_BAD_REQUEST
    assert rel(got[:2], ref[:2]) <= TOL["bf16"]


def test_attn_offsets_past_32_bits(torch):  # noqa: F811
    """A cache of more than 2^32 bytes, with a request in its first and last pages."""
    import serving_gdn_decode_gb300 as gdn
    c = Case(torch, "bf16", [40], n_kv=2, group=2, dim=256, page=16, extra=0)
    n_pages = (1 << 32) // (2 * 16 * 256) + 40
    big = [torch.full((n_pages, 2, 16, 256), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = [torch.full((n_pages, 2), math.nan, device="cuda") for _ in range(2)]
    at = torch.tensor([n_pages - 1, 0, n_pages - 3])
    pages = c.table[0].long().cpu()
    for i in range(2):
        big[i][at.cuda()] = c.cache_dev[i].view(torch.uint8)[pages.cuda()]
        scale[i][at.cuda()] = c.scale_dev[i][pages.cuda()]
    ref = c.reference(torch)
    c.table[0] = at.int().cuda()
    c.cache_dev, c.scale_dev = [b.view(torch.float8_e4m3fn) for b in big], scale
    assert rel(c.run(torch), ref) <= TOL["bf16"]
    # store to and load from the last page
    k, v = (torch.randn(2, 2, 256, generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2))
    slots = torch.tensor([n_pages * 16 - 2, n_pages * 16 - 1], dtype=torch.int32, device="cuda")
    gdn.gdn_kv_store_fp8(k, v, slots, *c.cache_dev, *c.scale_dev)
    k2, v2 = torch.empty_like(k), torch.empty_like(v)
    gdn.gdn_kv_load_fp8(slots, *c.cache_dev, *c.scale_dev, k2, v2)
    torch.cuda.synchronize()
    for x, y, sc in ((k, k2, scale[0]), (v, v2, scale[1])):
        # half a step of a code, or of the smallest codes (2^-9 of the page's scale apart)
        assert bool(((x - y).abs() <= x.abs() * 2.0 ** -4 + sc[-1][None, :, None] * 2.0 ** -10).all())
    assert bool((big[0][1:5] == 0x7F).all())


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page,dim,group", [(16, 64, 4), (24, 128, 2), (8, 256, 1)])
def test_steps_together(torch, dtype, page, dim, group):  # noqa: F811
    """Plan, store, attention and load over six steps with a rollback: the cache holds what was stored, each step's
    attention is that over the values which the cache stands for."""
    import serving_gdn_decode_gb300 as gdn
    n_kv, n_seqs, n_pages, max_pages = 2, 4, 60, 24
    dt = dtype_of(torch, dtype)
    dev = dict(dtype=torch.int32, device="cuda")
    i32 = lambda *s: torch.zeros(*s, **dev)  # noqa: E731
    cache = [torch.full((n_pages, n_kv, page, dim), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    scale = [torch.full((n_pages, n_kv), math.nan, device="cuda") for _ in range(2)]
    table, free = torch.full((n_seqs, max_pages), -1, **dev), torch.arange(n_pages, **dev)
    ctx, owned, n_free = i32(n_seqs), i32(n_seqs), torch.full((1,), n_pages, **dev)
    g = torch.Generator().manual_seed(9)
    held = [[[], []] for _ in range(n_seqs)]  # the requests' k and v rows
    for step, new in enumerate(([30, 1, 0, 17], [1, 1, 1, 1], [4, 3, 2, 1], [1, 1, 0, 1], [2, 2, 2, 2], [1, 1, 1, 1])):
        if step == 3:  # two drafted tokens of request 0 are refused
            ctx[0] -= 2
            for rows in held[0]:
                del rows[-2:]
        t = sum(new)
        kv_lens, owned_out, n_free_out, start = i32(n_seqs), i32(n_seqs), i32(1), i32(n_seqs + 1)
        slots, positions = i32(t), i32(t)
        gdn.gdn_kv_plan(ctx, torch.tensor(new, **dev), owned, free, n_free, table, page, n_pages, kv_lens, owned_out,
                        n_free_out, start, slots, positions)
        size = 2.0 ** step if step % 2 else 1.0  # later tokens larger: scales grow
        k, v = (size * torch.randn(2, t, n_kv, dim, generator=g)).to(dt).cuda()
        gdn.gdn_kv_store_fp8(k, v, slots, *cache, *scale)
        q = torch.randn(t, n_kv * group, dim, generator=g).to(dt).cuda()
        out = torch.empty_like(q)
        ws = torch.empty(gdn.gdn_attn_fp8_workspace_size(q, cache[0], n_seqs), dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_paged_fp8(q, *cache, *scale, table, kv_lens, start, out, ws, scale=0.25 / math.sqrt(dim))
        ctx, owned, n_free = kv_lens, owned_out, n_free_out
        row = 0
        ref = torch.zeros(q.shape, dtype=torch.float64)
        for s, w in enumerate(new):
            for rows, x in zip(held[s], (k, v)):
                rows += list(x[row : row + w].double().cpu())
            n = len(held[s][0])
            at = torch.tensor([int(table[s, j // page]) * page + j % page for j in range(n)], **dev)
            back = [torch.empty(n, n_kv, dim, device="cuda") for _ in range(2)]
            gdn.gdn_kv_load_fp8(at, *cache, *scale, *back)
            torch.cuda.synchronize()
            for rows, got, sc in zip(held[s], back, scale):
                if n:
                    want = torch.stack(rows)
                    # each rounding on the way is half a step: one when it was stored, one each time the scale grew
                    # (exact but for the smallest codes)
                    small = sc[at.long() // page].double().cpu()[:, :, None] * 2.0 ** -9
                    assert bool(((got.double().cpu() - want).abs() <= want.abs() * 2.0 ** -4 + small).all())
            for i in range(w):
                hi = n - w + i + 1
                kk, vv = (b[:hi].double().cpu().permute(1, 0, 2) for b in back)
                qq = q[row].double().cpu().view(n_kv, group, dim)
                p = torch.softmax(0.25 / math.sqrt(dim) * torch.einsum("hgd,hkd->hgk", qq, kk), -1)
                ref[row] = torch.einsum("hgk,hkd->hgd", p, vv).reshape(-1, dim)
                row += 1
        assert rel(out, ref) <= TOL[dtype]
