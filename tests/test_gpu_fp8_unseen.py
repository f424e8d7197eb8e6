"""GPU tests of gdn_attn_paged_fp8: what a row does not see may hold anything.  Tolerances are those of test_gpu_fp8.py."""
import math

import pytest

from test_gpu_fp8 import TOL, Case, rel
from test_gpu_paged import clean_status, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu

SCALES = [-math.inf, math.inf, math.nan, -3.0e38, -1.0, 0.0]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group", [(64, 4), (128, 4), (128, 9), (128, 20), (256, 4), (256, 14)])
@pytest.mark.parametrize("page", [8, 12, 16])
@pytest.mark.parametrize("scale", SCALES)
def test_attn_any_scale_behind_the_window(torch, dtype, dim, group, page, scale):  # noqa: F811
    """Pages behind every row's window in a tile of which rows see other pages."""
    c = Case(torch, dtype, [150, 90, 33], wins=[3, 1, 2], dim=dim, group=group, page=page, n_kv=1)
    for window in (17, 33, 40):
        ref = c.reference(torch, window=window)
        keep = [x.clone() for x in c.scale_dev]
        for s, (n, w) in enumerate(zip(c.lens, c.wins)):
            for j in range(max(0, n - w + 1 - window) // page):
                for x in c.scale_dev:
                    x[int(c.table[s, j])] = scale
        got = c.run(torch, window=window)
        for x, y in zip(c.scale_dev, keep):
            x.copy_(y)
        assert rel(got, ref) <= TOL[dtype]
    assert status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim,group,page", [(64, 4, 24), (128, 4, 12), (128, 20, 20), (256, 4, 12)])
@pytest.mark.parametrize("scale", SCALES)
def test_attn_any_scale_of_a_page_of_none(torch, dtype, dim, group, page, scale):  # noqa: F811
    """The first page of the cache, which no request has, with requests that end inside a tile."""
    lens = [29, 61, 5, 130]
    seed = next(i for i in range(99) if not (Case(torch, dtype, lens, n_kv=1, group=1, dim=dim, page=page, seed=i).table == 0).any())
    c = Case(torch, dtype, lens, wins=[1, 3, 1, 2], n_kv=2, group=group, dim=dim, page=page, seed=seed)
    for x in c.scale_dev:
        x[0] = scale
    c.check(torch, dtype)
    assert status() == 0
