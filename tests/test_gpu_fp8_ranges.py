"""GPU tests of the 8-bit paged cache beyond single calls and over long ranges:
streams and graphs, a million keys, many short requests, prompts among decodes,
alignments.  Tolerances are those of test_gpu_fp8.py, with what is said at a test.
"""
import math

import numpy as np
import pytest

from test_gpu_fp8 import TOL, Case, Store, dtype_of, nearest, same
from test_gpu_paged import clean_status, rel, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,group", [(64, 2), (64, 12), (64, 30), (128, 4), (128, 12), (128, 30), (256, 8), (256, 12), (256, 30)])
def test_attn_sums_of_long_items_do_not_drift(torch, dim, group):  # noqa: F811
    """A million keys per request and requests enough that few are split: values of mean 1.5 show any leaning of the
    running sums' roundings.

    The one rounding of the result is below 2^-9 root-mean-square of an element, independent from column to column (each
    has a mean of its own): the mean signed error over `dim` columns stays below 4 * 2^-9 / sqrt(dim), four standard
    deviations.  A probability's rounding, 2^-12 root-mean-square, averages over a million keys; a tile's 16 or 32 products
    are summed in the tensor cores, which cut up to 2 bits below f32's 24 toward zero: 2^-22; f32 sums rounded to nearest
    add 2^-24 * sqrt(2^16): all within TOL's 2e-5."""
    import serving_gdn_decode_gb300 as gdn
    n, page, n_req = 1 << 20, 1024, 320
    g = torch.Generator(device="cuda").manual_seed(dim + group)
    rand = lambda f, *s: f(*s, device="cuda", generator=g)  # noqa: E731
    e4m3 = torch.float8_e4m3fn
    k = rand(torch.randn, n // page, 1, page, dim).to(e4m3)
    v = (64.0 * (1.0 + rand(torch.rand, dim) + 0.5 * (rand(torch.rand, n // page, 1, page, dim) - 0.5))).to(e4m3)
    scale = [torch.exp2(torch.randint(-1, 2, (n // page, 1), device="cuda", generator=g).float()) for _ in range(2)]
    scale[1] /= 64.0
    q = rand(torch.randn, n_req, group, dim).to(torch.bfloat16)
    out = torch.empty_like(q)
    table = torch.arange(n // page, dtype=torch.int32, device="cuda")[None].repeat(n_req, 1).contiguous()  # one cache for all
    lens = torch.full((n_req,), n, dtype=torch.int32, device="cuda")
    ws = torch.empty(gdn.gdn_attn_fp8_workspace_size(q, k, n_req), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_paged_fp8(q, k, v, *scale, table, lens, None, out, ws)
    kk, vv = ((c.double() * s.double()[:, :, None, None]).reshape(-1, dim) for c, s in ((k, scale[0]), (v, scale[1])))
    for r in (0, 201, n_req - 1):
        p = torch.softmax(q[r].double() @ kk.T / math.sqrt(dim), -1)
        ref = p @ vv
        assert rel(out[r], ref) <= TOL["bf16"]
        signed = float(((out[r].double() - ref) / ref).mean())
        assert abs(signed) <= 4 * 2.0 ** -9 / math.sqrt(dim)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 16), (64, 24), (128, 24), (256, 16)])
def test_attn_many_short_requests(torch, dtype, dim, page):  # noqa: F811
    """More items than CTAs many times over, of one tile or less each, some without a key: the ring of jobs turns often."""
    r = np.random.RandomState(dim + page)
    lens = r.randint(0, 60, 1500)
    lens[r.randint(0, 1500, 200)] = 0
    Case(torch, dtype, lens.tolist(), n_kv=2, group=2, dim=dim, page=page).check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 8), (256, 2)])
@pytest.mark.parametrize("window", [0, 50])
def test_attn_prompts_among_decodes(torch, dtype, dim, group, window):  # noqa: F811
    Case(torch, dtype, [130, 77, 300, 90, 41], wins=[130, 1, 1, 33, 41], dim=dim, group=group, n_kv=1).check(torch, dtype, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,wins", [(16, (1, 1, 1)), (32, (1, 1, 1)), (40, (1, 1, 1)), (8, (7, 1, 4))])
@pytest.mark.parametrize("page", [24, 32])
def test_attn_wide_rows_over_long_keys(torch, dtype, dim, group, wins, page):  # noqa: F811
    """Blocks of 16 and 32 rows, split and joined."""
    c = Case(torch, dtype, [9001, 2000, 64], wins=wins, n_kv=1, group=group, dim=dim, page=page)
    c.check(torch, dtype)
    c.check(torch, dtype, window=300)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 3), (128, 20), (256, 2)])
def test_attn_q_aligned_to_four_bytes_only(torch, dtype, dim, group):  # noqa: F811
    c = Case(torch, dtype, [500, 33, 90], n_kv=2, group=group, dim=dim)
    a = c.run(torch).clone()
    pad = 2 if dtype == "bf16" else 1
    wide = torch.zeros(3, c.q.shape[1] * dim + pad, dtype=c.q.dtype, device="cuda")
    view = wide[:, pad:].unflatten(1, (c.q.shape[1], dim))
    view.copy_(c.q_dev)
    c.q_dev = view
    assert c.q_dev.data_ptr() % 16 != 0
    assert torch.equal(c.run(torch), a)


@pytest.mark.parametrize("dim,group,page", [(128, 4, 16), (128, 12, 24), (256, 8, 16), (64, 20, 8)])
def test_attn_a_page_that_one_row_sees_must_be_there(torch, dim, group, page):  # noqa: F811
    """A table entry that is none of the cache's makes all rows of the request NaN where the last token sees it alone; one
    behind every row's window nothing."""
    from serving_gdn_decode_gb300 import _native as nat
    c = Case(torch, "bf16", [4 * page + 1, 150], wins=[3, 2], n_kv=2, group=group, dim=dim, page=page)
    ref = c.reference(torch, window=2 * page)
    c.table[0, 0] = 1 << 30
    got = c.run(torch, window=2 * page)
    assert rel(got, ref) <= TOL["bf16"] and status() == 0
    c.table[0, 4] = -1
    got = c.run(torch, window=2 * page)
    assert status() == nat.GDN_DEVICE_BAD_PAGE
    assert bool(got[:3].isnan().all()) and rel(got[3:], ref[3:]) <= TOL["bf16"]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attn_large_values(torch, dtype):  # noqa: F811
    """Values of up to 2^90 and down to 2^-100."""
    for by in (2.0 ** 80, 2.0 ** -95):
        c = Case(torch, dtype, [700, 45], group=3, spread=0)
        c.scale[1] = c.scale[1] * by
        c.scale_dev[1].copy_(c.scale[1])
        c.check(torch, dtype)


def test_calls_on_two_streams(torch):  # noqa: F811
    """Calls that overlap on two streams, each with its own workspace, and calls back to back on one stream that share
    one, give what they give alone, bit for bit; stores and loads among them."""
    import serving_gdn_decode_gb300 as gdn
    cases = [Case(torch, "bf16", [3000 + 500 * i, 700, 64], dim=128, group=4, seed=i) for i in range(4)]
    alone = [c.run(torch).clone() for c in cases]
    for c in cases:
        c.out.fill_(9.0)
    size = max(gdn.gdn_attn_fp8_workspace_size(c.q_dev, c.cache_dev[0], 3) for c in cases)
    streams = [torch.cuda.Stream() for _ in range(2)]
    work = [torch.full((size,), 77, dtype=torch.uint8, device="cuda") for _ in range(2)]
    stores = [Store(torch, "bf16", range(5, 60), dim=128, seed=i) for i in range(2)]
    refs = [s.reference() for s in stores]
    slots = torch.arange(5, 60, dtype=torch.int32, device="cuda")
    back = [torch.empty(2, 55, 2, 128, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate(cases):
            gdn.gdn_attn_paged_fp8(c.q_dev, *c.cache_dev, *c.scale_dev, c.table, c.kv_lens, c.start, c.out, work[i % 2],
                                   stream=streams[i % 2])
            s = stores[i % 2]
            gdn.gdn_kv_store_fp8(s.k, s.v, slots, *s.cache, *s.scale, stream=streams[i % 2])
            gdn.gdn_kv_load_fp8(slots, *s.cache, *s.scale, *back[i % 2], stream=streams[i % 2])
    torch.cuda.synchronize()
    for c, want in zip(cases, alone):
        assert torch.equal(c.out, want)
    for s, (cache, scale), b in zip(stores, refs, back):
        for i in range(2):
            same(torch, s.cache[i], cache[i])
            same(torch, s.scale[i], scale[i])
            at = slots.long().cpu()
            same(torch, b[i], cache[i][at // 16, :, at % 16] * scale[i][at // 16][:, :, None])


def test_captured_steps(torch):  # noqa: F811
    """Plan, store, attention and load of a decode step captured once and replayed, the lengths growing on the device:
    the same as the steps run as they are, bit for bit."""
    import serving_gdn_decode_gb300 as gdn
    n_seqs, n_kv, group, dim, page, n_pages, max_pages = 3, 2, 4, 128, 16, 40, 12
    dev = dict(dtype=torch.int32, device="cuda")

    def serve(captured):
        i32 = lambda *s: torch.zeros(*s, **dev)  # noqa: E731
        cache = [torch.zeros(n_pages, n_kv, page, dim, device="cuda").to(torch.float8_e4m3fn) for _ in range(2)]
        scale = [torch.zeros(n_pages, n_kv, device="cuda") for _ in range(2)]
        table, free = torch.full((n_seqs, max_pages), -1, **dev), torch.arange(n_pages, **dev)
        ctx, owned, n_free = i32(n_seqs), i32(n_seqs), torch.full((1,), n_pages, **dev)
        kv_lens, owned_out, n_free_out, start, slots, pos = i32(n_seqs), i32(n_seqs), i32(1), i32(n_seqs + 1), i32(n_seqs), i32(n_seqs)
        new = torch.ones(n_seqs, **dev)
        rows = torch.randn(40, n_seqs, (group + 2) * n_kv, dim, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
        qkv = torch.empty_like(rows[0])
        q, k, v = (t.contiguous() for t in qkv.split([group * n_kv, n_kv, n_kv], 1))
        out, back = torch.empty_like(q), torch.empty(2, n_seqs, n_kv, dim, device="cuda")
        ws = torch.empty(gdn.gdn_attn_fp8_workspace_size(q, cache[0], n_seqs), dtype=torch.uint8, device="cuda")

        def step():
            for t, x in zip((q, k, v), qkv.split([group * n_kv, n_kv, n_kv], 1)):
                t.copy_(x)
            gdn.gdn_kv_plan(ctx, new, owned, free, n_free, table, page, n_pages, kv_lens, owned_out, n_free_out, start, slots, pos)
            gdn.gdn_kv_store_fp8(k, v, slots, *cache, *scale)
            gdn.gdn_attn_paged_fp8(q, *cache, *scale, table, kv_lens, start, out, ws)
            gdn.gdn_kv_load_fp8(slots, *cache, *scale, *back)
            for a, b in ((ctx, kv_lens), (owned, owned_out), (n_free, n_free_out)):
                a.copy_(b)

        graph, seen = None, []
        for i in range(40):
            qkv.copy_(rows[i] * 2.0 ** (i % 5))
            if captured and i >= 1:
                if graph is None:
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph):
                        step()
                graph.replay()
            else:
                step()
            seen.append((out.clone(), back.clone()))
        torch.cuda.synchronize()
        return seen, cache, scale

    a, ca, sa = serve(False)
    b, cb, sb = serve(True)
    for (x, y), (z, w) in zip(a, b):
        assert torch.equal(x, z) and torch.equal(y, w)
    for x, y in zip(ca + sa, cb + sb):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [64, 100])
def test_store_of_many_requests(torch, dtype, page):  # noqa: F811
    """Decodes and prompts in one call, more than the teams take at once, pages in any order."""
    r = np.random.RandomState(page)
    slots, used = [], 0
    order = r.permutation(1200)
    for _ in range(700):
        a, n = int(r.randint(0, page)), 1 if r.rand() < 0.9 else int(r.randint(1, 3 * page))
        for j in range(n):
            slots.append(int(order[used + (a + j) // page]) * page + (a + j) % page)
        used += (a + n - 1) // page + 1
        if used > 1100:
            break
    s = Store(torch, dtype, slots, n_pages=1200, page=page, dim=64, n_kv=1)
    first = [c.double().cpu() for c in s.cache], [x.double().cpu() for x in s.scale]
    s.call()
    at = torch.tensor(slots)
    p, o = at // page, at % page
    for i, x in enumerate((s.k, s.v)):
        x, scale = x.double().cpu()[:, 0], s.scale[i].double().cpu()[:, 0]
        top = torch.zeros(1200, dtype=torch.float64).scatter_reduce_(0, p, x.abs().amax(1), "amax")
        begins = torch.full((1200,), page).scatter_reduce_(0, p, o, "amin")
        m, e = torch.frexp(top)
        want = 2.0 ** (e - 9 + (m > 0.875).long()).double()
        want = torch.where(begins > 0, torch.maximum(want, first[1][i][:, 0]), want)
        touched = torch.zeros(1200, dtype=torch.bool)
        touched[p] = True
        assert torch.equal(scale, torch.where(touched, want, first[1][i][:, 0]))
        now = s.cache[i].double().cpu()[:, 0]
        same(torch, now[p, o], nearest(torch, x / want[p][:, None]))
        # the pages' earlier codes on the new scale; everything else untouched
        grown = nearest(torch, first[0][i][:, 0] * (first[1][i] / torch.where(touched, want, 1.0)[:, None])[:, :, None])
        place = torch.arange(page)[None, :]
        stored = torch.zeros(1200, page, dtype=torch.bool)
        stored[p, o] = True
        earlier = touched[:, None] & (place < begins[:, None]) & (want > first[1][i][:, 0])[:, None]
        same(torch, now[~stored], torch.where(earlier[:, :, None], grown, first[0][i][:, 0])[~stored])


@pytest.mark.parametrize("dtype,dim,n_kv,page", [("bf16", 128, 8, 64), ("bf16", 64, 8, 100), ("f32", 256, 8, 64)])
def test_store_of_prompts_between_decodes(torch, dtype, dim, n_kv, page):  # noqa: F811
    """Thousands of tokens, so that a team looks at more than 32 of them: prompts that begin and end inside pages, hundreds of
    decodes in a row, idle tokens among them."""
    r = np.random.RandomState(dim + page)
    order, used, slots = r.permutation(500), 0, []
    for n in [1] * 150 + [2500, 1, 1700, 2 * page] + [1] * 120 + [1111] + [1, 5] * 20:
        a = int(r.randint(0, page))
        slots += [int(order[used + (a + j) // page]) * page + (a + j) % page for j in range(n)] + [-1] * int(r.randint(0, 2))
        used += (a + n - 1) // page + 1
    Store(torch, dtype, slots, n_pages=500, page=page, dim=dim, n_kv=n_kv).check()


def test_hybrid_example_over_an_fp8_cache(torch, capsys):  # noqa: F811
    """The example's decode steps (captured and replayed) end where one pass over all tokens does.  Both hold the same
    values in 8 bits but for those that f32's roundings, which differ between the two, bring over a border of the codes,
    and the smallest of pages whose scale grew: far fewer than all, which would be 2^-4 of the attention's part."""
    from serving_gdn_decode_gb300 import hybrid_step
    assert hybrid_step.main(["--requests", "5", "--prompt", "37", "--steps", "20", "--cache", "fp8", "--check"]) <= 2.0 ** -4
    assert "device status 0" in capsys.readouterr().out
