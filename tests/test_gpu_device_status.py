"""GPU tests of gdn_device_status: what it costs, and that every file's word is in it."""
import threading
import time

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as t
    assert t.cuda.is_available(), "GPU tests need a CUDA device"
    from serving_gdn_decode_gb300 import build
    build.build()
    return t


def median_us(f, n=300):
    for _ in range(20):
        f()
    times = []
    for _ in range(n):
        t = time.perf_counter()
        f()
        times.append(time.perf_counter() - t)
    return sorted(times)[n // 2] * 1e6


def test_device_status_is_one_copy(torch):
    """However many files have a word: a read costs at most three times what reading one number off the device
    does (a launch, a copy and two waits), with the clearing too."""
    from serving_gdn_decode_gb300 import _native as nat
    x = torch.zeros(1, dtype=torch.int32, device="cuda")
    one = median_us(lambda: x.item())
    for reset in (False, True):
        assert median_us(lambda: nat.gdn_device_status(reset=reset)) <= 3 * one


def report(torch, gdn, bit):
    """A call that sets one bit."""
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    if bit == 2:  # a page more than the stack has
        gdn.gdn_kv_plan(i32(0), i32(9), i32(0), i32(1), i32(1), torch.full((1, 4), -1, dtype=torch.int32, device="cuda"), 8, 4,
                        i32(0), i32(0), i32(0), i32(0, 0), i32(*[0] * 9), i32(*[0] * 9))
    elif bit == 4:  # a negative length
        q, k = f(1, 1, 64), f(1, 1, 8, 64)
        ws = torch.empty(gdn.gdn_attn_workspace_size(q, k, 1), dtype=torch.uint8, device="cuda")
        gdn.gdn_attn_paged(q, k, k, i32(0)[None], i32(-1), None, f(1, 1, 64), ws)
    else:  # a position past the table
        gdn.gdn_rope(f(1, 1, 64), f(1, 1, 64), i32(7), f(4, 64), f(1, 1, 64), f(1, 1, 64))


def test_device_status_gathers_every_word(torch):
    import serving_gdn_decode_gb300 as gdn
    from serving_gdn_decode_gb300 import _native as nat
    nat.gdn_device_status(reset=True)
    for bits in ((2,), (4,), (16,), (2, 4, 16)):
        for b in bits:
            report(torch, gdn, b)
        torch.cuda.synchronize()
        assert nat.gdn_device_status() == sum(bits)  # reading keeps them
        assert nat.gdn_device_status(reset=True) == sum(bits)
        assert nat.gdn_device_status() == 0


def test_device_status_from_several_threads(torch):
    """Each of the bits set is given out by exactly one of the clearing reads that go on meanwhile."""
    import serving_gdn_decode_gb300 as gdn
    from serving_gdn_decode_gb300 import _native as nat
    nat.gdn_device_status(reset=True)
    stop, seen, errors = threading.Event(), [], []

    def read(stream):
        try:
            while not stop.is_set():
                bits = nat.gdn_device_status(reset=True, stream=stream)
                if bits:
                    seen.append(bits)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=read, args=(torch.cuda.Stream(),)) for _ in range(3)]
    for t in threads:
        t.start()
    rounds = 30
    for _ in range(rounds):
        report(torch, gdn, 16)
        torch.cuda.synchronize()
        time.sleep(0.005)
    stop.set()
    for t in threads:
        t.join()
    left = nat.gdn_device_status(reset=True)
    assert not errors
    assert len(seen) + (left == 16) == rounds and set(seen) <= {16}
