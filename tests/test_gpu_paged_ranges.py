"""GPU tests of the full-attention operators over ranges that test_gpu_paged.py does not
reach, against plain implementations in 64 bits; its tolerances, and per request or row
where one request could hide another's error.
"""
import math

import pytest

from test_gpu_paged import TOL, Case, clean_status, dtype_of, rel, torch  # noqa: F401 (fixtures among them)

pytestmark = pytest.mark.gpu


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
