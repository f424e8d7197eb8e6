"""GPU tests of gdn_attn_paged_fp8 over pages of 8 tokens, of whole groups of 8 and of others, with few and many rows per key
head: rows one by one and in boxes, in blocks of 8, 16 and 32 rows.  Tolerances are those of test_gpu_fp8.py."""
import pytest

from test_gpu_fp8 import Case
from test_gpu_paged import clean_status, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("group", [8, 9, 17, 40])
@pytest.mark.parametrize("page", [4, 8, 12, 20, 24, 40])
def test_attn_rows_and_pages(torch, dtype, dim, group, page):  # noqa: F811
    c = Case(torch, dtype, [300, 5, 77, 1500], wins=[1, 2, 1, 1], dim=dim, group=group, n_kv=1, page=page)
    c.check(torch, dtype)
    c.check(torch, dtype, window=50)
    assert status() == 0
