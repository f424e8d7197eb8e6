"""GPU tests of gdn_attn_paged_fp8 where its inner waits run out: the limit is set so low that warps give up on copies and
partners that are merely not there yet.  Every row is then right, NaN, or not written; the status says so; and the calls after
it are as ever."""
import pytest

from test_gpu_fp8 import Case
from test_gpu_paged import clean_status, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [4, 12, 30])
@pytest.mark.parametrize("page", [16, 24])
def test_attn_waits_that_run_out(torch, dtype, dim, group, page):  # noqa: F811
    from serving_gdn_decode_gb300 import _native as nat
    cases = [Case(torch, dtype, [9001, 700, 64, 0], wins=[2, 1, 3, 1], n_kv=1, group=group, dim=dim, page=page),
             Case(torch, dtype, [40 + 3 * i for i in range(70)], n_kv=2, group=group, dim=dim, page=page, seed=1)]
    right = [c.run(torch).clone() for c in cases]
    assert status() == 0
    some = 0
    try:
        for clocks in (1, 100, 500, 1000, 2000, 3000, 5000, 8000, 15000):
            nat.gdn_attn_fp8_wait_clocks(clocks)
            for c, want in zip(cases, right):
                c.out.fill_(7.0)
                got = c.run(torch).flatten(0, 1)  # a row per token and head
                st = status()
                want = want.flatten(0, 1)
                good = (got == want).all(1)
                lost = got.isnan().all(1) | (got == 7.0).all(1)
                assert bool((good | lost).all())
                assert st == (0 if good.all() else nat.GDN_DEVICE_WAIT_TIMEOUT) or (good.all() and st == nat.GDN_DEVICE_WAIT_TIMEOUT)
                some += int(not good.all())
    finally:
        nat.gdn_attn_fp8_wait_clocks(0)
    assert some  # at one clock hardly anything is there
    for c, want in zip(cases, right):
        c.out.fill_(7.0)
        assert torch.equal(c.run(torch), want)
    assert status() == 0
