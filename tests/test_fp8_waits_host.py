"""The limit of gdn_attn_paged_fp8's inner waits as the C ABI takes it (no GPU needed)."""
import pytest

from serving_gdn_decode_gb300 import _native as nat
from test_paged_host import L  # noqa: F401


def test_wait_clocks(L):  # noqa: F811
    assert L.gdn_attn_fp8_wait_clocks((1 << 31) + 1) == nat.GDN_ERR_INVALID_ARGUMENT
    assert "2^31" in nat.gdn_last_error()
    for clocks in (1, 1 << 31, 0):
        assert L.gdn_attn_fp8_wait_clocks(clocks) == nat.GDN_OK and nat.gdn_last_error() == ""
    for clocks in ((1 << 31) + 1, (1 << 32) - 1, 1 << 32, (1 << 32) + 5, -1):
        with pytest.raises(nat.GdnError, match="2\\^31"):
            nat.gdn_attn_fp8_wait_clocks(clocks)
    nat.gdn_attn_fp8_wait_clocks()
