"""GPU tests of the 8-bit cache's store in pages of very many tokens."""
import pytest

from test_gpu_fp8 import nearest, same
from test_gpu_paged import clean_status, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu


def test_store_past_2_27_tokens_of_a_page(torch):  # noqa: F811
    """A page of more than 2^31 pieces of 16 codes before the stored run (34 GB each for k and v): where its scale grows all
    codes before are rounded again, those at its beginning and past 2^31 pieces alike."""
    import serving_gdn_decode_gb300 as gdn
    dim, place = 256, (1 << 27) + 40
    free = torch.cuda.mem_get_info()[0]
    if free < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    cache = [torch.zeros(1, 1, place + 64, dim, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator().manual_seed(1)
    at = [0, 1, 7, 12345, 1 << 26, (1 << 27) - 1, 1 << 27, (1 << 27) + 1, place - 1]
    codes = (torch.randn(len(at), dim, generator=g) * 60).to(torch.float8_e4m3fn)
    for c in cache:
        c[0, 0, at] = codes.view(torch.uint8).cuda()
    scale = [torch.full((1, 1), 2.0 ** -3, device="cuda") for _ in range(2)]
    k, v = (x * torch.randn(64, 1, dim, generator=g).to(torch.bfloat16).cuda() for x in (4096.0, 1.0))  # k's scale grows, v's not
    slots = torch.arange(place, place + 64, dtype=torch.int32, device="cuda")
    gdn.gdn_kv_store_fp8(k, v, slots, *(c.view(torch.float8_e4m3fn) for c in cache), *scale)
    torch.cuda.synchronize()
    need = 2.0 ** -3
    while float(k.abs().max()) > 448 * need:
        need *= 2
    assert need > 2.0 ** -3 and float(scale[0]) == need and float(scale[1]) == 2.0 ** -3
    now = [c[0, 0, at].view(torch.float8_e4m3fn) for c in cache]
    same(torch, now[0], nearest(torch, codes.double() * (2.0 ** -3 / need)))
    same(torch, now[1], codes)
    for c, x, s in zip(cache, (k, v), (need, 2.0 ** -3)):
        same(torch, c[0, 0, place:].view(torch.float8_e4m3fn), nearest(torch, x[:, 0].double().cpu() / s))
    assert status() == 0
    del cache
    torch.cuda.empty_cache()
