"""Cases for the operators of a full-attention layer in a hybrid model's serving
step: the layer that stands next to the Gated DeltaNet layers this package runs.

* plan -- block table, slot map, positions and lengths of one step, made on the
  GPU from the request lengths;
* rope -- rotary positions with several axes on q and k, and the store of k and
  v in the paged cache;
* attn -- attention of each request's newest tokens over its paged cache.

``run`` computes a case in plain torch operations (``own`` false) or through
the package's entry points (``own`` true).
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One decode step of a small batch: every request adds one token, few need a page.
        {"name": "plan_decode", "op": "plan", "seqs": 64, "ctx_max": 4096, "new": "one",
         "new_max": 1, "page": 16, "lens_seed": 1},
        # A server's mixed step at full load: mostly decodes, some prompts of up to 4096 tokens.
        {"name": "plan_mixed", "op": "plan", "seqs": 1024, "ctx_max": 16384, "new": "mixed",
         "new_max": 4096, "page": 16, "lens_seed": 2},
        # Decode batch of 64 requests: one token each, text positions.
        {"name": "rope_decode", "op": "rope", "kind": "store", "dtype": "bf16", "tokens": 64,
         "n_q": 32, "n_kv": 8, "dim": 128, "rot": 128, "axes": 1, "interleaved": False, "page": 16},
        # Prefill of 4 x 4096 tokens, text and image patches mixed: time, height and width axes.
        {"name": "rope_prefill", "op": "rope", "kind": "store", "dtype": "bf16", "tokens": 16384,
         "n_q": 32, "n_kv": 8, "dim": 128, "rot": 128, "axes": 3, "interleaved": False, "page": 16},
        # A short f32 prompt with a partial rotation (64 of 256 dims) of neighbouring pairs.
        {"name": "rope_partial", "op": "rope", "kind": "store", "dtype": "f32", "tokens": 333,
         "n_q": 16, "n_kv": 2, "dim": 256, "rot": 64, "axes": 3, "interleaved": True, "page": 32},
        # Training of an image encoder: the rotation of the gradients of q and k (no cache), two axes.
        {"name": "rope_gradient", "op": "rope", "kind": "inverse", "dtype": "bf16", "tokens": 8209,
         "n_q": 16, "n_kv": 16, "dim": 64, "rot": 64, "axes": 2, "interleaved": False, "page": 16},
        # One user, one new token, a short context: latency.
        {"name": "attn_one", "op": "attn", "dtype": "bf16", "seqs": 1, "ctx_max": 1021, "window_tokens": 1,
         "n_q": 16, "n_kv": 2, "dim": 256, "page": 16, "sliding": 0, "lens_seed": 3},
        # A decode batch of 64 requests with contexts of up to 4096 tokens, some slots of the batch idle.
        {"name": "attn_decode", "op": "attn", "dtype": "bf16", "seqs": 64, "ctx_max": 4096,
         "window_tokens": 1, "n_q": 32, "n_kv": 8, "dim": 128, "page": 16, "sliding": 0, "lens_seed": 4},
        # A wide decode batch of 256 requests: throughput.
        {"name": "attn_wide", "op": "attn", "dtype": "bf16", "seqs": 256, "ctx_max": 4096,
         "window_tokens": 1, "n_q": 48, "n_kv": 8, "dim": 128, "page": 64, "sliding": 0, "lens_seed": 5},
        # One request over a very long document: only a split over the length fills the GPU.
        {"name": "attn_long", "op": "attn", "dtype": "bf16", "seqs": 1, "ctx_max": 200003,
         "window_tokens": 1, "n_q": 32, "n_kv": 4, "dim": 128, "page": 16, "sliding": 0, "lens_seed": 6},
        # Speculative verification: windows of 1 to 4 drafted tokens on 32 requests.
        {"name": "attn_verify", "op": "attn", "dtype": "bf16", "seqs": 32, "ctx_max": 8191,
         "window_tokens": 4, "n_q": 16, "n_kv": 2, "dim": 256, "page": 32, "sliding": 0, "lens_seed": 7},
        # f32 activations and cache, one key head per query head, sliding window of 1000 keys.
        {"name": "attn_f32", "op": "attn", "dtype": "f32", "seqs": 24, "ctx_max": 2500, "window_tokens": 1,
         "n_q": 16, "n_kv": 16, "dim": 64, "page": 16, "sliding": 1000, "lens_seed": 8},
    ]


#: Most bf16 cache elements (padded to the longest request) and row elements a drawn case holds, after the largest listed ones.
MOST_CACHE, MOST_ROPE = 256 * 4096 * 8 * 128 // 2, 16384 * 48 * 128


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "rope", "attn", "attn", "attn"])
    if op == "plan":
        new = rng.choice(["one", "mixed"])
        return {"op": op, "seqs": _log(rng, 1, 1024), "ctx_max": _log(rng, 16, 16384), "new": new,
                "new_max": 1 if new == "one" else _log(rng, 2, 4096),
                "page": rng.choice([1, 8, 16, 24, 32, 64, 128]), "lens_seed": rng.randrange(1 << 30)}
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    n_kv, group, dim = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 6, 8]), rng.choice([64, 128, 256])
    page = rng.choice([8, 16, 24, 32, 64, 128])
    if op == "rope":
        kind = rng.choice(["store", "store", "forward", "inverse"])
        most = max(1, MOST_ROPE * 2 // SIZE[dtype] // ((group + 2) * n_kv * dim))
        return {"op": op, "kind": kind, "dtype": dtype, "tokens": _log(rng, 1, min(most, 32768)),
                "n_q": n_kv * group, "n_kv": n_kv, "dim": dim, "rot": rng.choice([dim, dim, dim // 2, dim // 4]),
                "axes": rng.choice([1, 2, 3, 4]), "interleaved": rng.random() < 0.3, "page": page}
    seqs, window = _log(rng, 1, 256), rng.choice([1, 1, 1, 2, 4, 7])
    most = max(16, MOST_CACHE * 2 // SIZE[dtype] // (seqs * n_kv * dim * max(1, window * group // 32)))
    return {"op": op, "dtype": dtype, "seqs": seqs, "ctx_max": _log(rng, 16, min(most, 200000)),
            "window_tokens": window, "n_q": n_kv * group, "n_kv": n_kv, "dim": dim,
            "page": page, "sliding": rng.choice([0, 0, 0, 128, 1000]), "lens_seed": rng.randrange(1 << 30)}


# ------------------------------------------------------------------ sizes of a case


def _plan_lens(case):
    """Cached and new tokens of each request: contexts uniform up to ctx_max; "one": a token each,
    one slot in 16 idle; "mixed": one request in 16 a prompt (log-uniform length, no context)."""
    r = np.random.RandomState(case["lens_seed"] % (1 << 31))
    n = case["seqs"]
    ctx = r.randint(0, case["ctx_max"] + 1, n)
    new = (r.randint(0, 16, n) > 0).astype(np.int64)
    if case["new"] == "mixed":
        prompt = r.randint(0, 16, n) == 0
        prompt[0] = True
        length = np.exp(r.uniform(0, math.log(case["new_max"]), n)).round().astype(np.int64)
        length[0] = case["new_max"]
        ctx, new = np.where(prompt, 0, ctx), np.where(prompt, length, new)
    else:
        new[0] = 1
    return ctx.astype(np.int64), new.astype(np.int64)


def _attn_lens(case):
    """Cached tokens (the window among them) and window of each request: lengths uniform up to ctx_max,
    the first at ctx_max, one in 16 an idle slot with neither; windows of 1 to window_tokens."""
    r = np.random.RandomState(case["lens_seed"] % (1 << 31))
    n = case["seqs"]
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


def _visible(case):
    """For each request: keys that at least one of its tokens sees, and (token, key) pairs seen."""
    kv, win = _attn_lens(case)
    w = case["sliding"] or (1 << 40)
    keys = np.where(win > 0, np.minimum(kv, w + win - 1), 0)
    pairs = sum(np.where(t < win, np.maximum(0, np.minimum(kv - win + t + 1, w)), 0) for t in range(case["window_tokens"]))
    return keys, pairs


def work(case):
    if case["op"] == "plan":
        ctx, new = _plan_lens(case)
        pages = np.maximum(0, -(-(ctx + new) // case["page"]) - (-(-ctx // case["page"]))).sum()
        ints = 3 * len(ctx) + 1 + pages  # lengths, owned pages, free pages
        ints += pages + 2 * len(ctx) + 1 + len(ctx) + 1 + 2 * new.sum()  # table entries, lengths, starts, slots, positions
        return {"bytes": 4 * int(ints), "flops": 0}
    if case["op"] == "rope":
        t, n_q, n_kv, d, rot = (case[k] for k in ("tokens", "n_q", "n_kv", "dim", "rot"))
        store = case["kind"] == "store"
        elems = t * d * (n_q + n_kv * (2 if store else 1))
        extra = 4 * t * (case["axes"] + (1 if store else 0)) + 4 * rot * min(t, _table_rows(case))
        return {"bytes": 2 * elems * SIZE[case["dtype"]] + extra, "flops": 3 * t * (n_q + n_kv) * rot}
    keys, pairs = _visible(case)
    _, win = _attn_lens(case)
    d, es = case["dim"], SIZE[case["dtype"]]
    b = 2 * int(keys.sum()) * case["n_kv"] * d * es + 2 * int(win.sum()) * case["n_q"] * d * es
    b += 4 * int(_attn_pages(case).sum()) + 8 * case["seqs"] + 4
    return {"bytes": b, "flops": 4 * int(pairs.sum()) * case["n_q"] * d}


def _table_rows(case):
    return max(4096, case["tokens"])


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"plan": _prepare_plan, "rope": _prepare_rope, "attn": _prepare_attn}[case["op"]](case, g)
    return {"case": dict(case), **state}


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _table(pages, width, pool):
    """Block table of -1 with request s's first pages[s] entries taken from `pool` in order."""
    pages = torch.from_numpy(np.ascontiguousarray(pages)).cuda()
    cols = torch.arange(width, device="cuda")[None, :]
    held = cols < pages[:, None]
    at = (pages.cumsum(0) - pages)[:, None] + cols
    return torch.where(held, pool[torch.where(held, at, 0)], -1).to(torch.int32).contiguous()


def _prepare_plan(case, g):
    ctx, new = _plan_lens(case)
    page, n = case["page"], case["seqs"]
    owned, need = -(-ctx // page), -(-(ctx + new) // page)
    width = int(need.max()) + 1
    n_pages = int(need.sum()) + 64
    pool = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    free = pool[int(owned.sum()):].contiguous()
    slots = int(new.sum()) + 13  # a fixed capacity a little over the step's tokens
    e = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")  # noqa: E731
    return {"ctx_lens": _ints(ctx), "new_lens": _ints(new), "owned": _ints(owned), "free_pages": free,
            "n_free": _ints([free.numel()]), "block_table": _table(owned, width, pool), "n_pages": n_pages,
            "kv_lens": e(n), "owned_out": e(n), "n_free_out": e(1), "token_start": e(n + 1),
            "slot_map": e(slots), "positions": e(slots)}


def _prepare_rope(case, g):
    t, n_q, n_kv, d, rot, axes = (case[k] for k in ("tokens", "n_q", "n_kv", "dim", "rot", "axes"))
    dt, page, store = DTYPES[case["dtype"]], case["page"], case["kind"] == "store"
    # q, k and v as the fused projection of a layer leaves them: views of one row per token
    qkv = torch.randn(t, (n_q + 2 * n_kv) * d, generator=g, device="cuda").to(dt)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([n_q * d, n_kv * d, n_kv * d], 1))
    rows = _table_rows(case)
    freq = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * freq
    table = torch.cat([angle.cos(), angle.sin()], 1).float()
    # runs of text (all axes alike) and of image patches (a 32-wide grid)
    i = torch.arange(t, device="cuda")
    at = torch.randint(0, rows - t + 1, (1,), generator=g, device="cuda") + i
    image = (i // 256) % 2 == 1
    grid = [i // 256 * 256 + at[0] - i[0], (i % 256) // 32, i % 32, at % 7]
    pos = torch.stack([torch.where(image & (axes > 1), grid[a] % rows, at) for a in range(axes)]).to(torch.int32)
    state = {"q": q, "k": k, "v": v, "positions": pos, "cos_sin": table,
             "axes": bytes((j * axes) // (rot // 2) for j in range(rot // 2)),
             "q_out": torch.zeros(t, n_q, d, dtype=dt, device="cuda")}
    if store:
        n_pages = -(-t // page) + 3
        pages = torch.randperm(n_pages, generator=g, device="cuda")
        slots = pages[i // page] * page + i % page
        state["slot_map"] = torch.where(i % 61 == 60, -1, slots).to(torch.int32)  # padding tokens have no slot
        for name in ("k_cache", "v_cache"):
            state[name] = torch.randn(n_pages, n_kv, page, d, generator=g, device="cuda").to(dt)
    else:
        state["k_out"] = torch.zeros(t, n_kv, d, dtype=dt, device="cuda")
    return state


def _prepare_attn(case, g):
    kv, win = _attn_lens(case)
    pages = _attn_pages(case)
    n_pages = int(pages.sum()) + 5
    dt, d = DTYPES[case["dtype"]], case["dim"]
    n = int(win.sum())
    pool = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    shape = (n_pages, case["n_kv"], case["page"], d)
    state = {"q": 2.0 * torch.randn(n, case["n_q"], d, generator=g, device="cuda").to(dt),
             "k_cache": torch.randn(shape, generator=g, device="cuda", dtype=dt),
             "v_cache": torch.randn(shape, generator=g, device="cuda", dtype=dt),
             "block_table": _table(pages, int(pages.max()), pool), "kv_lens": _ints(kv),
             "token_start": _ints(np.concatenate([[0], np.cumsum(win)])),
             "output": torch.zeros(n, case["n_q"], d, dtype=dt, device="cuda")}
    if own:  # the workspace a server keeps beside its cache
        from serving_gdn_decode_gb300 import gdn_attn_workspace_size
        size = gdn_attn_workspace_size(state["q"], state["k_cache"], case["seqs"])
        state["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return state


# ------------------------------------------------------------------ one pass


def run(state):
    op = state["case"]["op"]
    if own:
        return {"plan": _own_plan, "rope": _own_rope, "attn": _own_attn}[op](state)
    return {"plan": _plain_plan, "rope": _plain_rope, "attn": _plain_attn}[op](state)


_PLAN_OUT = ("block_table", "kv_lens", "owned_out", "n_free_out", "token_start", "slot_map", "positions")


def _own_plan(s):
    import serving_gdn_decode_gb300 as gdn
    gdn.gdn_kv_plan(s["ctx_lens"], s["new_lens"], s["owned"], s["free_pages"], s["n_free"], s["block_table"],
                    s["case"]["page"], s["n_pages"], s["kv_lens"], s["owned_out"], s["n_free_out"],
                    s["token_start"], s["slot_map"], s["positions"])
    return {k: s[k] for k in _PLAN_OUT}


def _own_rope(s):
    import serving_gdn_decode_gb300 as gdn
    kind, inter = s["case"]["kind"], s["case"]["interleaved"]
    if kind == "store":
        gdn.gdn_rope_store(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slot_map"], s["k_cache"],
                           s["v_cache"], s["q_out"], axes=s["axes"], interleaved=inter)
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    gdn.gdn_rope(s["q"], s["k"], s["positions"], s["cos_sin"], s["q_out"], s["k_out"], axes=s["axes"],
                 interleaved=inter, inverse=kind == "inverse")
    return [s["q_out"], s["k_out"]]


def _own_attn(s):
    import serving_gdn_decode_gb300 as gdn
    gdn.gdn_attn_paged(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["kv_lens"], s["token_start"],
                       s["output"], s["workspace"], window=s["case"]["sliding"])
    return s["output"]


def _plain_plan(s):
    page = s["case"]["page"]
    ctx, new, owned = s["ctx_lens"].long(), s["new_lens"].long(), s["owned"].long()
    table, slots = s["block_table"], s["slot_map"]
    need = torch.maximum(owned, (ctx + new + page - 1) // page)
    demand = need - owned
    base = demand.cumsum(0) - demand
    served = base + demand <= s["n_free"]
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (cols >= owned[:, None]) & (cols < need[:, None]) & served[:, None]
    rank = torch.where(fresh, s["n_free"] - 1 - (base[:, None] + cols - owned[:, None]), 0)
    table.copy_(torch.where(fresh, s["free_pages"][rank], table))
    end = new.cumsum(0)
    start = end - new
    i = torch.arange(slots.numel(), device=table.device)
    seq = torch.searchsorted(end, i, right=True)
    real = seq < new.numel()
    seq = torch.where(real, seq, 0)
    pos = ctx[seq] + i - start[seq]
    held = real & served[seq]
    slot = table[seq, torch.where(held, pos // page, 0)] * page + pos % page
    slots.copy_(torch.where(held, slot, -1))
    s["positions"].copy_(torch.where(real, pos, 0))
    s["kv_lens"].copy_(torch.where(served, ctx + new, ctx))
    s["owned_out"].copy_(torch.where(served, need, owned))
    s["n_free_out"].copy_(s["n_free"] - torch.where(served, demand, 0).sum())
    s["token_start"][0] = 0
    s["token_start"][1:] = end
    return {k: s[k] for k in _PLAN_OUT}


def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2 : rot]
    c, d = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    case = s["case"]
    rot, half, inter = case["rot"], case["rot"] // 2, case["interleaved"]
    axis = torch.tensor(list(s["axes"]), device=s["q"].device)
    pos = s["positions"][axis].t().long()  # [tokens, pairs]
    pair = torch.arange(half, device=pos.device)
    cos, sin = s["cos_sin"][pos, pair][:, None], s["cos_sin"][pos, half + pair][:, None]
    if case["kind"] == "inverse":
        sin = -sin
    s["q_out"].copy_(_rotate(s["q"], cos, sin, rot, inter))
    k = _rotate(s["k"], cos, sin, rot, inter)
    if case["kind"] != "store":
        s["k_out"].copy_(k)
        return [s["q_out"], s["k_out"]]
    keep = s["slot_map"] >= 0
    slot = s["slot_map"][keep].long()
    page, at = slot // case["page"], slot % case["page"]
    s["k_cache"][page, :, at] = k[keep].to(s["k_cache"].dtype)
    s["v_cache"][page, :, at] = s["v"][keep]
    return [s["q_out"], s["k_cache"], s["v_cache"]]


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
    k = s["k_cache"][table].transpose(1, 2).reshape(n_seqs, n_kv, length, d).float()
    score = q @ k.transpose(2, 3) * (1.0 / math.sqrt(d))
    del k
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
    v = s["v_cache"][table].transpose(1, 2).reshape(n_seqs, n_kv, length, d).float()
    v = torch.where(held, v, 0.0)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    out = out.view(n_seqs, n_kv, t_max, group, d).permute(0, 2, 1, 3, 4).reshape(n_seqs, t_max, case["n_q"], d)
    s["output"].copy_(out[real])
    return s["output"]


# ------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(case, s)
    half, inter = case["rot"] // 2, case["interleaved"]
    sign = -1.0 if case["kind"] == "inverse" else 1.0
    turned = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for j in range(half):
            at = s["positions"][s["axes"][j]].long()
            c, n = s["cos_sin"][at, j].double()[:, None], sign * s["cos_sin"][at, half + j].double()[:, None]
            a, b = (2 * j, 2 * j + 1) if inter else (j, j + half)
            y[..., a] = x[..., a].double() * c - x[..., b].double() * n
            y[..., b] = x[..., b].double() * c + x[..., a].double() * n
        turned.append(y)
    if case["kind"] != "store":
        return turned
    caches = [s["k_cache"].double(), s["v_cache"].double()]
    for cache, rows in zip(caches, (turned[1], s["v"].double())):
        flat = cache.transpose(1, 2).reshape(-1, case["n_kv"], case["dim"])
        for i, slot in enumerate(s["slot_map"].tolist()):
            if slot >= 0:
                flat[slot] = rows[i]
        cache.copy_(flat.view(cache.shape[0], case["page"], case["n_kv"], case["dim"]).transpose(1, 2))
    return [turned[0], *caches]


def _exact_attn(case, s):
    kv, win = _attn_lens(case)
    group = case["n_q"] // case["n_kv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for i, (n, w) in enumerate(zip(kv.tolist(), win.tolist())):
        if not w:
            continue
        pages = s["block_table"][i, : -(-n // case["page"])].long()
        k, v = (s[name][pages].double().permute(1, 0, 2, 3).reshape(case["n_kv"], -1, case["dim"])[:, :n]
                for name in ("k_cache", "v_cache"))
        for t in range(w):
            hi = n - w + t + 1
            lo = max(0, hi - case["sliding"]) if case["sliding"] else 0
            q = s["q"][row].double().view(case["n_kv"], group, case["dim"])
            p = torch.softmax(torch.einsum("hgd,hkd->hgk", q, k[:, lo:hi]) / math.sqrt(case["dim"]), -1)
            out[row] = torch.einsum("hgk,hkd->hgd", p, v[:, lo:hi]).reshape(case["n_q"], case["dim"])
            row += 1
    return out
