"""GPU tests of gdn_attn_paged_fp8 where a row's probabilities and its pages' scales differ widely, against plain
implementations in 64 bits.  Tolerances are those of test_gpu_fp8.py; far below the maximum a probability times its value's
scale is good to 2^-31 (f32: 2^-35) of the row's largest such product, which over these tests' 256 keys and codes of at most
448 against a mean of 64 stays below 2^-31 * 2^8 * 2^3 = 2^-20: within TOL's 2e-5.
"""
import math

import numpy as np
import pytest

from test_gpu_fp8 import TOL, TOP, Case, rel
from test_gpu_paged import clean_status, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


SCORE = math.log(2.0) * 5 * 2.0 ** -24


def check(c, torch, dtype, bits, **kw):  # noqa: F811
    ref, got = c.reference(torch, **kw), c.run(torch, **kw).double().cpu()
    tol = TOL[dtype] + bits * SCORE
    assert rel(got, ref) <= tol
    assert float(((got - ref).norm(dim=-1) / ref.norm(dim=-1)).max()) <= 3 * tol


def upload(c, torch):  # noqa: F811
    for i in range(2):
        c.cache_dev[i].view(torch.uint8).copy_(c.codes(torch, i))
        c.scale_dev[i].copy_(c.scale[i])
    c.q_dev.copy_(c.q)


def weighted(torch, dtype, lens, small, bits, wins=None, **kw):  # noqa: F811
    """A case in which the keys that `small(request, key)` names have probabilities of 2^-bits of the others' or a little
    more: a key's score is its element 0."""
    c = Case(torch, dtype, lens, wins=wins, n_kv=1, spread=0, **kw)
    c.q.zero_()
    c.q[..., 0] = 8.0
    r = np.random.RandomState(bits)
    c.cache[0] *= 0.0  # scores of 0, and NaN where there is no key
    for s, n in enumerate(c.lens):
        keys = np.array([j for j in range(n) if small(s, j)], dtype=np.int64)
        pages = c.table[s].cpu().numpy()[keys // c.page]
        c.cache[0][pages, 0, keys % c.page, 0] = torch.tensor(r.choice([-448.0, -416.0, -384.0], len(keys))).float()
    c.scale[0] *= bits * math.log(2.0) * math.sqrt(c.dim) / (8.0 * TOP) / c.scale[0]
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,page", [(2, 16), (2, 24), (2, 64), (12, 32), (30, 16)])
@pytest.mark.parametrize("bits", [20, 28, 34, 38, 60, 100])
def test_attn_small_probabilities_of_large_values(torch, dtype, dim, group, page, bits):  # noqa: F811
    """Every part of the kernel meets keys of large probability first; then come keys of probabilities 2^-bits of theirs in
    pages whose values are 2^bits times as large, or more."""
    c = weighted(torch, dtype, [256, 250], lambda s, j: j >= 128 or j % 16 != 0, bits, dim=dim, group=group, page=page)
    small = c.scale[1].clone()
    for more in (0, 10):
        c.scale[1] = small.clone()
        for s in range(2):
            for j in range(128 // page, -(-c.lens[s] // page)):
                if j * page >= 128:
                    c.scale[1][int(c.table[s, j])] *= 2.0 ** (bits + more)
        upload(c, torch)
        check(c, torch, dtype, bits)
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group,page", [(2, 8), (2, 12), (12, 8), (30, 16)])
@pytest.mark.parametrize("bits", [20, 34, 60])
def test_attn_small_probabilities_beside_large_ones(torch, dtype, dim, group, page, bits):  # noqa: F811
    """Pages of large probabilities and small values, and of small ones and large values, in turn: both in one tile of the
    kernel.  Windows of tokens: the last keys are seen by some rows only."""
    wins = [3, 1] if group < 12 else [1, 2]
    c = weighted(torch, dtype, [256, 77], lambda s, j: j // page % 2 == 1, bits, wins=wins, dim=dim, group=group, page=page)
    for s in range(2):
        for j in range(1, -(-c.lens[s] // page), 2):
            c.scale[1][int(c.table[s, j])] *= 2.0 ** bits
    upload(c, torch)
    check(c, torch, dtype, bits)
    check(c, torch, dtype, bits, window=100)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nats", [11, 14, 17, 20])
def test_attn_tails_of_equal_probabilities(torch, dtype, nats):  # noqa: F811
    """Tens of thousands of keys `nats` below one key in 64 whose value is zero, so that the small ones make the result: each is
    good to TOL's share of it or 2^-36 of the largest, all in the same direction at worst."""
    n, page = 60001, 64
    bits = nats / math.log(2.0)
    c = Case(torch, dtype, [n], n_kv=1, group=3, dim=128, page=page, spread=0)
    c.q.zero_()
    c.q[..., 0] = 8.0
    c.cache[0] *= 0.0
    c.cache[0][:, 0, 1:, 0] -= TOP
    c.scale[0] *= nats * math.sqrt(c.dim) / (8.0 * TOP) / c.scale[0]
    c.cache[1] = (c.cache[1] + 64.0).to(torch.float8_e4m3fn).float()
    c.cache[1][:, :, 0] = 0.0
    upload(c, torch)
    assert rel(c.run(torch), c.reference(torch)) <= TOL[dtype] + bits * SCORE + 2.0 ** (bits - 36)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group,page", [(64, 4, 16), (64, 12, 24), (128, 4, 16), (128, 12, 16), (128, 30, 32), (256, 2, 24), (256, 12, 16)])
def test_attn_large_queries_of_small_keys(torch, dtype, dim, group, page):  # noqa: F811
    """Queries near the largest values against key scales near the smallest: neither is out of range, nor are the scores.  One
    head's queries stay small, so that its scores are about zero."""
    c = Case(torch, dtype, [100, 64, 33], wins=[3, 1, 1], group=group, dim=dim, page=page, spread=1)
    c.q = (c.q.double() * 2.0 ** 121).to(c.q.dtype)
    c.q[:, 1] = (c.q[:, 1].double() * 2.0 ** -150).to(c.q.dtype)
    c.scale[0] = (c.scale[0].double() * 2.0 ** -121).float()
    assert bool(c.q.isfinite().all()) and bool((c.scale[0] != 0).all())
    upload(c, torch)
    c.check(torch, dtype)
    c.q = (c.q.double() * 2.0 ** -200).to(c.q.dtype)  # and small ones against large keys
    c.scale[0] = (c.scale[0].double() * 2.0 ** 200).float()
    upload(c, torch)
    c.check(torch, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group,page", [(64, 4, 16), (64, 12, 8), (64, 30, 24), (128, 4, 12), (128, 12, 16), (128, 30, 8), (256, 2, 16), (256, 30, 24)])
@pytest.mark.parametrize("far", [0, 3, 12, 40])
def test_attn_scales_of_any_value(torch, dtype, dim, group, page, far):  # noqa: F811
    """Scales that are no powers of two, negative and zero, up to 2^far apart."""
    c = Case(torch, dtype, [700, 64, 33, 130], wins=[3, 1, 2, 1], group=group, dim=dim, page=page, spread=0, seed=far)
    g = torch.Generator().manual_seed(far + page)
    for i in range(2):
        s = c.scale[i]
        by = (0.5 + torch.rand(s.shape, generator=g)) * torch.sign(torch.rand(s.shape, generator=g) - 0.3)
        if i:
            by = by * torch.exp2(-(far * torch.rand(s.shape, generator=g)))
            by[torch.rand(s.shape, generator=g) < 0.05] = 0.0
        c.scale[i] = s * by
    upload(c, torch)
    check(c, torch, dtype, 35)
    check(c, torch, dtype, 35, window=100)
    assert status() == 0
