"""Host-side tests of what gdn_rope_store takes as caches (no GPU needed): rows of a cache
that share elements, and k and v caches that do, are refused; views of one array that only
lie among one another are not.

Calls pass made-up device addresses; one that is not refused fails at its launch, for want
of a device.
"""
import itertools
import random

import pytest

from serving_gdn_decode_gb300 import _native as nat
from test_abi_host import no_device
from test_paged_host import L, STORE, addresses, refused, rope  # noqa: F401 (L: fixture)


def taken(status):
    assert status == nat.GDN_ERR_CUDA, nat.gdn_last_error()


# rope's params there: bf16, 20 pages of 8 slots, 2 heads of 64; pages 1024, heads 512, slots 64 apart


@no_device
def test_rows_of_a_cache_must_not_overlap(L):  # noqa: F811
    for change in ({"cache_head_stride": 64}, {"cache_page_stride": 512}, {"cache_page_stride": 1023}, {"cache_head_stride": 448},
                   {"cache_slot_stride": 128}, {"cache_page_stride": 64, "cache_head_stride": 64}):
        assert refused(rope(L, True, change), "rows overlap") == nat.GDN_ERR_INVALID_ARGUMENT
    for change in ({}, {"cache_page_stride": 4096}, {"cache_head_stride": 64, "cache_slot_stride": 128},
                   {"cache_head_stride": 20 * 512, "cache_page_stride": 512},  # a pool of pages per head
                   {"n_pages": 1, "cache_page_stride": 64},                    # strides over one element say nothing
                   {"page_size": 1, "cache_slot_stride": 512}):
        taken(rope(L, True, change))


@no_device
def test_k_and_v_caches_must_not_share_rows(L):  # noqa: F811
    k = addresses(STORE)["k_cache"]
    for step in (64, 1, -64, 512, 1024, -1024, 19 * 1024, 63):  # in elements
        assert refused(rope(L, True, k_cache=k, v_cache=k + 2 * step), "v_cache overlaps k_cache") == nat.GDN_ERR_INVALID_ARGUMENT
    taken(rope(L, True, k_cache=k, v_cache=k + 2 * 20 * 1024))
    taken(rope(L, True, k_cache=k, v_cache=k - 2 * 20 * 1024))
    for view, step in (({"cache_page_stride": 2048}, 1024),                                        # pages of K and V in turn
                       ({"cache_page_stride": 2048}, 3 * 1024),                                    # with the next page's V
                       ({"cache_page_stride": 2048, "cache_head_stride": 1024, "cache_slot_stride": 128}, 64),  # slots
                       ({"cache_page_stride": 2048, "cache_head_stride": 1024}, 512)):             # heads
        taken(rope(L, True, view, k_cache=k, v_cache=k + 2 * step))
        refused(rope(L, True, view, k_cache=k, v_cache=k + 2 * (step + 2)), "v_cache overlaps k_cache")


@no_device
def test_cache_overlap_against_enumeration(L):  # noqa: F811
    r = random.Random(5)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        dim = r.choice([2, 4])
        ext = [r.randint(1, 4) for _ in range(3)]  # pages, heads, slots
        order = r.sample(range(3), 3)
        strides, span = [dim] * 3, dim
        for i in order:
            if ext[i] > 1:
                strides[i] = max(dim, span + r.choice([0, 0, 0, dim, 2 * dim, 1, -1, -dim]))
                span += (ext[i] - 1) * strides[i]
        step = r.choice([1, -1]) * r.randint(0, 2 * span)
        k = 1 << 35
        st = rope(L, True, {"head_dim": dim, "rot_dim": 2, "n_kv_heads": ext[1], "n_pages": ext[0], "page_size": ext[2],
                            "axes": [0], "cache_page_stride": strides[0], "cache_head_stride": strides[1],
                            "cache_slot_stride": strides[2]}, k_cache=k, v_cache=k + 2 * step)
        at = [sum(i * s for i, s in zip(ix, strides)) + e for ix in itertools.product(*map(range, ext)) for e in range(dim)]
        clean = len(set(at)) == len(at) and not set(at) & {a + step for a in at}
        nested, covered = True, dim
        for s, n in sorted((s, n) for s, n in zip(strides, ext) if n > 1):
            nested, covered = nested and s >= covered, covered + (n - 1) * s
        if clean and nested:
            taken(st)
        else:
            assert refused(st, "overlap") == nat.GDN_ERR_INVALID_ARGUMENT
        seen[clean] += 1
    assert min(seen.values()) > 400


def test_strides_over_one_element_make_no_layout(L):  # noqa: F811
    """A cache of one key head as it is and one whose heads and slots are swapped lie alike in memory (refused here
    for being on the host, after every other check)."""
    import torch

    from test_paged_host import call
    f = torch.zeros
    for k, v in ((f(5, 1, 8, 64), f(5, 8, 1, 64).transpose(1, 2)), (f(1, 2, 8, 64), f(3, 2, 8, 64)[:1].as_strided((1, 2, 8, 64), (7, 512, 64, 1)))):
        for op, more in (("attn_paged", {}), ("rope_store", dict(k=f(2, k.size(1), 64), v=f(2, k.size(1), 64)))):
            with pytest.raises(nat.GdnError, match="must be a CUDA tensor"):
                call(op, k_cache=k, v_cache=v, **more)
    with pytest.raises(nat.GdnError, match="one layout"):
        call("attn_paged", k_cache=f(5, 2, 8, 64), v_cache=f(5, 8, 2, 64).transpose(1, 2))
