"""GPU test of the example over an 8-bit cache, against the same steps with a plain store and plain attention.

Both hold the same values in the same codes and scales, but for values that the two f32 roundings upstream bring to either side
of a code's border.  Attention in f32 differs by 2e-5 at most (test_gpu_fp8.py); a code's step is 2^-4 of a value or more, so at
most 2e-5 * 2^4 = 3.2e-4 of the elements differ, by a step of 2^-3 of theirs at most: keys and values differ by
sqrt(3.2e-4) * 2^-3 = 2^-8.8 of their norm, the logits, in which attention is a part and values average over the keys, by less:
2^-8.  A page that stands for twice its values must be seen.
"""
import math

import pytest

from test_gpu_fp8 import least_scale, nearest
from test_gpu_paged import clean_status, status, torch  # noqa: F401

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -8


def plain_store(torch, k, v, slots, k_cache, v_cache, k_scale, v_scale):  # noqa: F811
    page = k_cache.shape[2]
    slots = slots.tolist()
    for p in dict.fromkeys(s // page for s in slots if s >= 0):
        rows = [i for i, s in enumerate(slots) if s >= 0 and s // page == p]
        a, n = slots[rows[0]] % page, len(rows)
        for c, sc, x in ((k_cache, k_scale, k), (v_cache, v_scale, v)):
            for h in range(c.shape[1]):
                y, old = x[rows, h].double().cpu(), float(sc[p, h])
                new = max(least_scale(float(y.abs().max())), old if a else 0.0)
                codes = c[p, h].double().cpu()
                codes[:a] = nearest(torch, codes[:a] * (old / new))
                codes[a : a + n] = nearest(torch, y / new)
                c[p, h] = codes.to(c.device).to(torch.float32).to(c.dtype)
                sc[p, h] = new


def plain_attention(torch, q, k_cache, v_cache, k_scale, v_scale, table, lens, start, out):  # noqa: F811
    page, dim = k_cache.shape[2:]
    n_kv, group = k_cache.shape[1], q.shape[1] // k_cache.shape[1]
    for s, n in enumerate(lens.tolist()):
        pages = table[s, : -(-n // page)].long()
        k, v = ((c[pages].double() * sc[pages].double()[:, :, None, None]).transpose(0, 1).reshape(n_kv, -1, dim)
                for c, sc in ((k_cache, k_scale), (v_cache, v_scale)))
        t0, t1 = start[s : s + 2].tolist()
        for t in range(t0, t1):
            hi = n - (t1 - t0) + (t - t0) + 1
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q[t].double().view(n_kv, group, dim), k[:, :hi]) / math.sqrt(dim), -1)
            out[t] = torch.einsum("hgk,hkd->hgd", p, v[:, :hi]).reshape(-1, dim).to(out.dtype)


def test_hybrid_example_against_plain_steps(torch, monkeypatch):  # noqa: F811
    from serving_gdn_decode_gb300 import hybrid_step
    requests, prompt, steps = 3, 37, 12
    model = hybrid_step.Model(hybrid_step.Config(cache="fp8"))
    prompts = torch.randint(0, model.cfg.vocab, (requests, prompt), generator=torch.Generator().manual_seed(1)).cuda()
    tokens, logits = hybrid_step.generate(model, prompts, steps)  # decode steps captured and replayed
    assert status() == 0
    monkeypatch.setattr(hybrid_step, "gdn_kv_store_fp8", lambda *a: plain_store(torch, *a))
    monkeypatch.setattr(hybrid_step, "gdn_attn_paged_fp8",
                        lambda q, kc, vc, ks, vs, table, lens, start, out, ws: plain_attention(torch, q, kc, vc, ks, vs, table, lens, start, out))

    def plain(spoil=None):
        server = hybrid_step.Server(model, requests, prompt, prompt + steps)
        server.step(prompts.reshape(-1), prompt)
        if spoil is not None:  # request 0's first page of the first layer's keys or values
            server.scales[0][spoil][int(server.table[0, 0])] *= 2
        for i in range(steps):
            out = server.step(tokens[:, i].contiguous(), 1)
        return ((logits.double() - out.double()).norm(dim=1) / out.double().norm(dim=1)).tolist()

    error = plain()
    print("logits against plain steps:", error)
    assert max(error) <= BOUND
    for spoil in (0, 1):
        spoilt = plain(spoil)
        print("with a page that stands for twice its values:", spoilt)
        assert spoilt[0] > 2 * BOUND and max(spoilt[1:]) <= BOUND
