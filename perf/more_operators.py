"""Cases for the 8-bit paged cache of a hybrid model's full-attention layers: the
same serving step as with a bf16 cache, with half the bytes per cached token.

* store -- a step's k and v quantised to e4m3 as they are written to the paged
  cache, with a power-of-two scale for each page and key head;
* load -- cached rows read back as values;
* attn -- attention of each request's newest tokens over the 8-bit cache.

``run`` computes a case in plain torch operations (``own`` false) or through
the package's entry points (``own`` true).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
MOST_CODE = 448.0  # the largest e4m3 value
LEAST, MOST = -110, 119  # exponents of a block's scale


def listed():
    return [
        # Decode step of 64 requests: one token each, appended somewhere in its page.
        {"name": "store_decode", "op": "store", "dtype": "bf16", "seqs": 64, "ctx_max": 4096, "new": "one",
         "new_max": 1, "n_kv": 8, "dim": 128, "page": 16, "lens_seed": 1},
        # Prefill of four prompts of about 4096 tokens, behind cached prefixes that end inside a page.
        {"name": "store_prefill", "op": "store", "dtype": "bf16", "seqs": 4, "ctx_max": 500, "new": "prompt",
         "new_max": 4096, "n_kv": 8, "dim": 128, "page": 64, "lens_seed": 2},
        # f32 activations, few wide heads, an odd page: a mixed step of decodes and short prompts.
        {"name": "store_mixed", "op": "store", "dtype": "f32", "seqs": 37, "ctx_max": 700, "new": "mixed",
         "new_max": 333, "n_kv": 2, "dim": 256, "page": 24, "lens_seed": 3},
        # Cached prefixes of 8 requests read back for a prefill that takes bf16 keys and values.
        {"name": "load_prefix", "op": "load", "dtype": "bf16", "seqs": 8, "ctx_max": 8191, "n_kv": 8, "dim": 128,
         "page": 16, "lens_seed": 4},
        # One short context handed on in f32.
        {"name": "load_short", "op": "load", "dtype": "f32", "seqs": 1, "ctx_max": 203, "n_kv": 16, "dim": 64,
         "page": 32, "lens_seed": 5},
        # One user, one new token, a short context: latency.
        {"name": "attn_one", "op": "attn", "dtype": "bf16", "seqs": 1, "ctx_max": 1021, "window_tokens": 1,
         "n_q": 16, "n_kv": 2, "dim": 256, "page": 16, "sliding": 0, "lens_seed": 6},
        # A decode batch of 64 requests with contexts of up to 4096 tokens, some slots of the batch idle.
        {"name": "attn_decode", "op": "attn", "dtype": "bf16", "seqs": 64, "ctx_max": 4096,
         "window_tokens": 1, "n_q": 32, "n_kv": 8, "dim": 128, "page": 16, "sliding": 0, "lens_seed": 7},
        # A wide decode batch of 256 requests: throughput.
        {"name": "attn_wide", "op": "attn", "dtype": "bf16", "seqs": 256, "ctx_max": 4096,
         "window_tokens": 1, "n_q": 48, "n_kv": 8, "dim": 128, "page": 64, "sliding": 0, "lens_seed": 8},
        # One request over a very long document: only a split over the length fills the GPU.
        {"name": "attn_long", "op": "attn", "dtype": "bf16", "seqs": 1, "ctx_max": 400009,
         "window_tokens": 1, "n_q": 32, "n_kv": 4, "dim": 128, "page": 16, "sliding": 0, "lens_seed": 9},
        # Speculative verification: windows of 1 to 4 drafted tokens on 32 requests.
        {"name": "attn_verify", "op": "attn", "dtype": "bf16", "seqs": 32, "ctx_max": 8191, "window_tokens": 4,
         "n_q": 16, "n_kv": 2, "dim": 256, "page": 32, "sliding": 0, "lens_seed": 10},
        # f32 activations, one key head per query head, sliding window of 1000 keys.
        {"name": "attn_f32", "op": "attn", "dtype": "f32", "seqs": 24, "ctx_max": 2500, "window_tokens": 1,
         "n_q": 16, "n_kv": 16, "dim": 64, "page": 16, "sliding": 1000, "lens_seed": 11},
        # Pages that end inside a tile: 24 tokens, heads of 64 in groups of three.
        {"name": "attn_odd", "op": "attn", "dtype": "bf16", "seqs": 40, "ctx_max": 3001, "window_tokens": 1,
         "n_q": 24, "n_kv": 8, "dim": 64, "page": 24, "sliding": 0, "lens_seed": 12},
    ]


#: Most cache elements (padded to the longest request) and row elements a drawn case holds, after the largest listed ones.
MOST_CACHE, MOST_ROWS = 256 * 4096 * 8 * 128, 4 * 4096 * 8 * 128


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "store", "load", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    n_kv, dim = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([64, 128, 256])
    page = rng.choice([8, 16, 16, 24, 32, 64, 128])
    case = {"op": op, "dtype": dtype, "n_kv": n_kv, "dim": dim, "page": page, "lens_seed": rng.randrange(1 << 30)}
    if op == "store":
        new = rng.choice(["one", "prompt", "mixed"])
        tokens = MOST_ROWS * 2 // SIZE[dtype] // (n_kv * dim)
        seqs = _log(rng, 1, min(tokens, 512 if new != "prompt" else 16))
        # of a mixed step, one request in 16 and one more is a prompt
        prompts = {"one": 1, "prompt": seqs, "mixed": seqs // 16 + 4}[new]
        new_max = 1 if new == "one" else _log(rng, 1, max(1, min(8192, (tokens - seqs) // prompts)))
        return {**case, "seqs": seqs, "ctx_max": _log(rng, 1, 16384), "new": new, "new_max": new_max}
    if op == "load":
        seqs = _log(rng, 1, 64)
        most = max(1, MOST_ROWS * 2 // SIZE[dtype] // (seqs * n_kv * dim))
        return {**case, "seqs": seqs, "ctx_max": _log(rng, 1, min(most, 65536))}
    group = rng.choice([1, 2, 3, 4, 6, 8])
    seqs, window = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4, 7])
    most = max(16, MOST_CACHE * 2 // SIZE[dtype] // (2 * seqs * n_kv * dim * max(1, window * group // 16)))
    return {**case, "seqs": seqs, "ctx_max": _log(rng, 16, min(most, 400000)), "window_tokens": window,
            "n_q": n_kv * group, "sliding": rng.choice([0, 0, 0, 128, 1000])}


# ------------------------------------------------------------------ sizes of a case


def _rand(case):
    return np.random.RandomState(case["lens_seed"] % (1 << 31))


def _store_lens(case):
    """Cached and new tokens of each request: contexts uniform up to ctx_max; "one": a token each, one slot
    in 16 idle; "prompt": new_max for the first, the others from half of it; "mixed": one request in 16 a prompt."""
    r, n, most = _rand(case), case["seqs"], case["new_max"]
    ctx = r.randint(0, case["ctx_max"] + 1, n)
    if case["new"] == "prompt":
        new = r.randint(max(1, most // 2), most + 1, n)
    else:
        new = (r.randint(0, 16, n) > 0).astype(np.int64)
        if case["new"] == "mixed":
            prompt = r.randint(0, 16, n) == 0
            new = np.where(prompt, r.randint(1, most + 1, n), new)
    new[0] = most
    return ctx.astype(np.int64), new.astype(np.int64)


def _store_slots(case):
    """Slot of each new token and the pages of the cache: each request's last cached page and its new ones."""
    ctx, new = _store_lens(case)
    page = case["page"]
    first = ctx // page  # the page of the first new token
    pages = np.where(new > 0, -(-(ctx + new) // page) - first, 0)
    n_pages = int(pages.sum()) + 3
    order = _rand(case).permutation(n_pages)
    base = np.cumsum(pages) - pages
    seq = np.repeat(np.arange(case["seqs"]), new)
    at = np.arange(new.sum()) - np.repeat(np.cumsum(new) - new, new) + ctx[seq]
    return order[base[seq] + at // page - first[seq]] * page + at % page, n_pages


def _load_lens(case):
    r = _rand(case)
    kv = r.randint(1, case["ctx_max"] + 1, case["seqs"])
    kv[0] = case["ctx_max"]
    return kv.astype(np.int64)


def _load_slots(case):
    """Slots of the requests' cached tokens, one after the other; one in 61 is padding."""
    kv, page = _load_lens(case), case["page"]
    pages = -(-kv // page)
    n_pages = int(pages.sum()) + 3
    order = _rand(case).permutation(n_pages)
    seq = np.repeat(np.arange(case["seqs"]), kv)
    at = np.arange(kv.sum()) - np.repeat(np.cumsum(kv) - kv, kv)
    slots = order[(np.cumsum(pages) - pages)[seq] + at // page] * page + at % page
    return np.where(np.arange(len(slots)) % 61 == 60, -1, slots), n_pages


def _attn_lens(case):
    """Cached tokens (the window among them) and window of each request: lengths uniform up to ctx_max,
    the first at ctx_max, one in 16 an idle slot with neither; windows of 1 to window_tokens."""
    r, n = _rand(case), case["seqs"]
    kv = r.randint(1, case["ctx_max"] + 1, n)
    win = r.randint(1, case["window_tokens"] + 1, n)
    idle = r.randint(0, 16, n) == 0
    idle[0] = False
    kv[0], win[0] = case["ctx_max"], case["window_tokens"]
    kv = np.maximum(kv, win)
    return np.where(idle, 0, kv).astype(np.int64), np.where(idle, 0, win).astype(np.int64)


def _attn_pages(case):
    kv, _ = _attn_lens(case)
    return -(-kv // case["page"])


def work(case):
    n_kv, d, es, page = case["n_kv"], case["dim"], SIZE[case["dtype"]], case["page"]
    if case["op"] in ("store", "load"):
        slots, _ = (_store_slots if case["op"] == "store" else _load_slots)(case)
        held = slots[slots >= 0]
        pages = len(np.unique(held // page))  # whose scales are written, or read
        return {"bytes": 2 * len(held) * n_kv * d * (es + 1) + 4 * len(slots) + 8 * pages * n_kv,
                "flops": 4 * len(held) * n_kv * d}
    kv, win = _attn_lens(case)
    w = case["sliding"] or (1 << 40)
    keys = np.where(win > 0, np.minimum(kv, w + win - 1), 0)  # that at least one token of the request sees
    pairs = sum(np.where(t < win, np.maximum(0, np.minimum(kv - win + t + 1, w)), 0) for t in range(case["window_tokens"]))
    pages = (-(-kv // page) - (kv - keys) // page).sum()
    b = 2 * int(keys.sum()) * n_kv * d + 8 * int(pages) * n_kv + 2 * int(win.sum()) * case["n_q"] * d * es
    b += 4 * int(pages) + 8 * case["seqs"] + 4
    return {"bytes": b, "flops": 4 * int(pairs.sum()) * case["n_q"] * d}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"store": _prepare_store, "load": _prepare_load, "attn": _prepare_attn}[case["op"]](case, g)
    return {"case": dict(case), **state}


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _channels(case, g):
    """Factors of a key's elements: a few channels of each head are several times larger, as in trained models."""
    f = torch.ones(case["n_kv"], case["dim"], device="cuda")
    large = torch.randint(0, case["dim"], (case["n_kv"], 4), generator=g, device="cuda")
    return f.scatter_(1, large, 6.0)


def _blocks(case, n_pages, factors, g):
    """Random pages held in 8 bits: codes [n_pages, n_kv, page, dim] and scales [n_pages, n_kv]."""
    n_kv, page, d = case["n_kv"], case["page"], case["dim"]
    codes = torch.empty(n_pages, n_kv, page, d, dtype=E4M3, device="cuda")
    scales = torch.empty(n_pages, n_kv, device="cuda")
    step = max(1, (1 << 28) // (n_kv * page * d))
    for p in range(0, n_pages, step):
        x = torch.randn(min(step, n_pages - p), n_kv, page, d, generator=g, device="cuda") * factors[:, None]
        scales[p : p + step] = _least_scale(x.abs().amax((2, 3)))
        codes[p : p + step] = (x / scales[p : p + step, :, None, None]).to(E4M3)
    return codes, scales


def _caches(case, n_pages, g):
    state = {}
    state["k_cache"], state["k_scale"] = _blocks(case, n_pages, _channels(case, g), g)
    state["v_cache"], state["v_scale"] = _blocks(case, n_pages, torch.ones(case["n_kv"], case["dim"], device="cuda"), g)
    return state


def _prepare_store(case, g):
    slots, n_pages = _store_slots(case)
    state = _caches(case, n_pages, g)  # what was cached before, and stale pages
    t, n_kv, d = len(slots), case["n_kv"], case["dim"]
    k = torch.randn(t, n_kv, d, generator=g, device="cuda") * _channels(case, g)
    # v as the fused projection of a layer leaves it: a view of one row per token
    kv = torch.randn(t, 2 * n_kv * d, generator=g, device="cuda").to(DTYPES[case["dtype"]])
    return {**state, "slot_map": _ints(slots), "k": k.to(DTYPES[case["dtype"]]),
            "v": kv[:, n_kv * d :].unflatten(1, (n_kv, d))}


def _prepare_load(case, g):
    slots, n_pages = _load_slots(case)
    e = lambda: torch.zeros(len(slots), case["n_kv"], case["dim"], dtype=DTYPES[case["dtype"]], device="cuda")  # noqa: E731
    return {**_caches(case, n_pages, g), "slot_map": _ints(slots), "k": e(), "v": e()}


def _prepare_attn(case, g):
    kv, win = _attn_lens(case)
    pages = _attn_pages(case)
    n_pages, n = int(pages.sum()) + 5, int(win.sum())
    state = _caches(case, n_pages, g)
    pool = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    held = torch.from_numpy(pages).cuda()
    cols = torch.arange(int(pages.max()), device="cuda")[None, :]
    at = (held.cumsum(0) - held)[:, None] + cols
    table = torch.where(cols < held[:, None], pool[torch.where(cols < held[:, None], at, 0)], -1)
    q = 1.5 * torch.randn(n, case["n_q"], case["dim"], generator=g, device="cuda")
    q = q.to(DTYPES[case["dtype"]])
    state |= {"q": q, "block_table": table.to(torch.int32).contiguous(), "kv_lens": _ints(kv),
              "token_start": _ints(np.concatenate([[0], np.cumsum(win)])), "output": torch.zeros_like(q)}
    if own:  # the workspace a server keeps beside its cache
        from serving_gdn_decode_gb300 import gdn_attn_fp8_workspace_size
        size = gdn_attn_fp8_workspace_size(q, state["k_cache"], case["seqs"])
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"store": _own_store, "load": _own_load, "attn": _own_attn}[op](state)
    return {"store": _plain_store, "load": _plain_load, "attn": _plain_attn}[op](state)


_CACHE = ("k_cache", "v_cache", "k_scale", "v_scale")


def _own_store(s):
    import serving_gdn_decode_gb300 as gdn
    gdn.gdn_kv_store_fp8(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
    return {name: s[name] for name in _CACHE}


def _own_load(s):
    import serving_gdn_decode_gb300 as gdn
    gdn.gdn_kv_load_fp8(s["slot_map"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["k"], s["v"])
    return [s["k"], s["v"]]


def _own_attn(s):
    import serving_gdn_decode_gb300 as gdn
    gdn.gdn_attn_paged_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_table"],
                           s["kv_lens"], s["token_start"], s["output"], s["workspace"], window=s["case"]["sliding"])
    return s["output"]


def _code(x):
    """The nearest e4m3 value; what is not finite becomes NaN."""
    return torch.where(x.isfinite(), x.clamp(-MOST_CODE, MOST_CODE), math.nan).to(E4M3)


def _least_scale(amax):
    """The smallest power of two s with amax <= 448 s, as f32."""
    m, e = torch.frexp(amax)  # m in [0.5, 1), 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875).int(), LEAST).clamp(LEAST, MOST)
    return ((e + 127) << 23).view(torch.float32)  # exactly 2^e


def _plain_store(s):
    page = s["case"]["page"]
    slot = s["slot_map"].long()
    at, place = slot // page, slot % page
    # runs of tokens whose slots follow one another in a page
    follows = (slot[1:] == slot[:-1] + 1) & (place[1:] > 0) & (slot[:-1] >= 0)
    first = torch.nn.functional.pad(~follows, (1, 0), value=True)
    run_of = first.long().cumsum(0) - 1
    starts = first.nonzero()[:, 0]
    held = slot >= 0
    live = held[starts]
    at_run, place_run = at[starts].clamp(min=0), torch.where(live, place[starts], 0)
    for name in ("k", "v"):
        x, cache, scales = s[name].float(), s[name + "_cache"], s[name + "_scale"]
        amax = torch.where(x.isfinite(), x.abs(), 0.0).amax(2)
        top = torch.zeros(len(starts), x.shape[1], device=x.device)
        top.scatter_reduce_(0, run_of[:, None].expand_as(amax), amax, "amax")
        need, old = _least_scale(top), scales[at_run]
        scale = torch.where((place_run > 0)[:, None], torch.maximum(old, need), need)
        # the pages that a run goes on with: rounded again where the scale has grown
        grown = (place_run > 0) & live
        earlier = torch.arange(page, device=x.device)[None, None, :, None] < place_run[grown][:, None, None, None]
        earlier = earlier & (scale > old)[grown][:, :, None, None]
        block = cache[at_run[grown]].float()
        block = torch.where(earlier, block * (old / scale)[grown][:, :, None, None], block)
        cache[at_run[grown]] = block.to(E4M3)
        cache[at[held], :, place[held]] = _code(x / scale[run_of][:, :, None])[held]
        scales[at_run[live]] = scale[live]
    return {name: s[name] for name in _CACHE}


def _plain_load(s):
    page = s["case"]["page"]
    held = (s["slot_map"] >= 0)[:, None, None]
    slot = s["slot_map"].clamp(min=0).long()
    for name in ("k", "v"):
        x = s[name + "_cache"][slot // page, :, slot % page].float() * s[name + "_scale"][slot // page][:, :, None]
        s[name].copy_(torch.where(held, x, s[name].float()))
    return [s["k"], s["v"]]


def _plain_attn(s):
    case = s["case"]
    n_kv, d, t_max = case["n_kv"], case["dim"], case["window_tokens"]
    group = case["n_q"] // n_kv
    table, kv, start = s["block_table"].clamp(min=0), s["kv_lens"].long(), s["token_start"].long()
    n_seqs, dev = kv.numel(), kv.device
    win = start[1:] - start[:-1]
    t = torch.arange(t_max, device=dev)[None, :]
    real = t < win[:, None]
    at = torch.where(real, start[:-1, None] + t, 0)
    q = s["q"][at].float().view(n_seqs, t_max, n_kv, group, d).permute(0, 2, 1, 3, 4)
    q = q.reshape(n_seqs, n_kv, t_max * group, d)
    length = table.shape[1] * case["page"]

    def rows(name):  # [n_seqs, n_kv, length, d]
        x = s[name + "_cache"][table].float() * s[name + "_scale"][table][..., None, None]
        return x.transpose(1, 2).reshape(n_seqs, n_kv, length, d)

    score = q @ rows("k").transpose(2, 3) * (1.0 / math.sqrt(d))
    last = (kv[:, None] - win[:, None] + t)[:, :, None]
    key = torch.arange(length, device=dev)[None, None, :]
    seen = (key <= last) & real[:, :, None]
    if case["sliding"]:
        seen = seen & (key > last - case["sliding"])
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, group, -1).reshape(n_seqs, 1, t_max * group, length)
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - torch.where(top.isinf(), 0.0, top)), 0.0)
    total = p.sum(-1, keepdim=True)
    held = (key[0, 0] < kv[:, None])[:, None, :, None]
    out = torch.where(total > 0, (p @ torch.where(held, rows("v"), 0.0)) / total, 0.0)
    out = out.view(n_seqs, n_kv, t_max, group, d).permute(0, 2, 1, 3, 4).reshape(n_seqs, t_max, case["n_q"], d)
    s["output"].copy_(out[real])
    return s["output"]


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "load": _exact_load, "attn": _exact_attn}[case["op"]](case, s)


def _nearest(y):
    """y (64 bits) on the grid of e4m3: steps of 2^(e - 3) from 2^e on, of 2^-9 below 2^-6; ties to even."""
    e = torch.frexp(y.abs().clamp(min=2.0 ** -6)).exponent.long() - 1
    step = (e - 3 + 1023 << 52).view(torch.float64)
    return (torch.round(y / step) * step).clamp(-MOST_CODE, MOST_CODE)


def _exact_store(case, s):
    page = case["page"]
    out = {name: s[name].double() for name in _CACHE}
    powers = torch.tensor([2.0 ** e for e in range(LEAST, MOST + 1)], dtype=torch.float64, device="cuda")
    slots = s["slot_map"].tolist()
    i = 0
    while i < len(slots):
        j = i + 1
        while j < len(slots) and slots[j] == slots[j - 1] + 1 and slots[j] % page:
            j += 1
        p, a = slots[i] // page, slots[i] % page
        for name in ("k", "v"):
            x = s[name][i:j].double().transpose(0, 1)  # [n_kv, tokens, dim]
            cache, scales = out[name + "_cache"], out[name + "_scale"]
            old = scales[p].clone()
            scale = powers[torch.searchsorted(MOST_CODE * powers, x.abs().amax((1, 2))).clamp(max=len(powers) - 1)]
            if a:
                scale = torch.maximum(scale, old)
                cache[p, :, :a] = _nearest(cache[p, :, :a] * (old / scale)[:, None, None])
            cache[p, :, a : a + j - i] = _nearest(x / scale[:, None, None])
            scales[p] = scale
        i = j
    return out


def _exact_load(case, s):
    out = [s["k"].double(), s["v"].double()]
    held = (s["slot_map"] >= 0).nonzero()[:, 0]
    p, at = s["slot_map"][held].long() // case["page"], s["slot_map"][held].long() % case["page"]
    for h in range(case["n_kv"]):
        for x, name in zip(out, ("k", "v")):
            x[held, h] = s[name + "_cache"][p, h, at].double() * s[name + "_scale"][p, h].double()[:, None]
    return out


def _exact_attn(case, s):
    kv, win = _attn_lens(case)
    group = case["n_q"] // case["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for i, (n, w) in enumerate(zip(kv.tolist(), win.tolist())):
        if not w:
            continue
        pages = s["block_table"][i, : -(-n // case["page"])].long()
        k, v = ((s[name + "_cache"][pages].double() * s[name + "_scale"][pages].double()[:, :, None, None])
                .permute(1, 0, 2, 3).reshape(case["n_kv"], -1, case["dim"])[:, :n] for name in ("k", "v"))
        for t in range(w):
            hi = n - w + t + 1
            lo = max(0, hi - case["sliding"]) if case["sliding"] else 0
            q = s["q"][row].double().view(case["n_kv"], group, case["dim"])
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q, k[:, lo:hi]) / math.sqrt(case["dim"]), -1)
            out[row] = torch.einsum("hgk,hkd->hgd", p, v[:, lo:hi]).reshape(case["n_q"], case["dim"])
            row += 1
    return out
