"""A small hybrid model served step by step: Gated DeltaNet layers and a
full-attention layer over a paged cache, with random weights.

Each block is three linear-attention layers (``gdn_forward``) and one
full-attention layer (``gdn_rope_store`` and ``gdn_attn_paged``); one
``gdn_kv_plan`` per step serves every attention layer.  The prompts go through as
one step of many tokens, then one token per request and step; the decode step
reads everything it needs from device memory, so it is captured once in a CUDA
graph and replayed::

    python -m serving_gdn_decode_gb300.hybrid_step --requests 16 --prompt 100 --steps 64

With ``--check`` the logits of the last step are compared with those of a model
that sees all tokens at once.
"""
from __future__ import annotations

import argparse
import math
from dataclasses import dataclass

import torch

from . import (gdn_attn_paged, gdn_attn_workspace_size, gdn_forward, gdn_kv_plan, gdn_rope_store,
               pack_params)


@dataclass(frozen=True)
class Config:
    blocks: int = 2
    gdn_per_block: int = 3
    width: int = 512
    gdn_dim: int = 64
    gdn_k_heads: int = 2
    gdn_v_heads: int = 4
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    rot_dim: int = 64
    vocab: int = 1024
    page: int = 16
    max_tokens: int = 4096


def rope_table(cfg: Config, device) -> torch.Tensor:
    freq = 10000.0 ** (-torch.arange(cfg.rot_dim // 2, dtype=torch.float64) * 2 / cfg.rot_dim)
    angle = torch.arange(cfg.max_tokens, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().to(device)


class Model:
    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        w = lambda n, m: (torch.randn(n, m, generator=g) / math.sqrt(n)).to(device)  # noqa: E731
        self.cfg, self.device = cfg, torch.device(device)
        self.embed = torch.randn(cfg.vocab, cfg.width, generator=g).to(device)
        self.head = w(cfg.width, cfg.vocab)
        dk, nk, nv = cfg.gdn_dim, cfg.gdn_k_heads, cfg.gdn_v_heads
        self.gdn = [dict(qkv=w(cfg.width, (2 * nk + nv) * dk), gates=w(cfg.width, 2 * nv), out=w(nv * dk, cfg.width))
                    for _ in range(cfg.blocks * cfg.gdn_per_block)]
        d, nq, nkv = cfg.head_dim, cfg.q_heads, cfg.kv_heads
        self.attn = [dict(qkv=w(cfg.width, (nq + 2 * nkv) * d), out=w(nq * d, cfg.width)) for _ in range(cfg.blocks)]
        self.table = rope_table(cfg, device)


class Server:
    """The state of `requests` requests of up to `tokens` tokens: recurrent states, the paged cache and its plan."""

    def __init__(self, model: Model, requests: int, prompt: int, tokens: int):
        cfg, dev, s = model.cfg, model.device, requests
        if tokens > cfg.max_tokens:  # past the table of cosines the rotated q and k would be NaN
            raise ValueError(f"{tokens} tokens per request, but the model has {cfg.max_tokens} positions")
        self.model, self.requests = model, s
        self.max_pages = -(-tokens // cfg.page)
        self.n_pages = s * self.max_pages
        i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device=dev)  # noqa: E731
        self.states = [torch.zeros(s * cfg.gdn_v_heads * cfg.gdn_dim ** 2, device=dev) for _ in model.gdn]
        shape = (self.n_pages, cfg.kv_heads, cfg.page, cfg.head_dim)
        self.caches = [(torch.zeros(shape, device=dev), torch.zeros(shape, device=dev)) for _ in model.attn]
        self.table = torch.full((s, self.max_pages), -1, dtype=torch.int32, device=dev)
        self.free = torch.arange(self.n_pages, dtype=torch.int32, device=dev)
        self.ctx, self.owned, self.n_free = i32(s), i32(s), torch.full((1,), self.n_pages, dtype=torch.int32, device=dev)
        self.kv_lens, self.owned_out, self.n_free_out, self.start = i32(s), i32(s), i32(1), i32(s + 1)
        self.by_width = {}  # per step width: buffers of the step, made once
        for width in (prompt, 1):
            q = torch.empty(s * width, cfg.q_heads, cfg.head_dim, device=dev)
            self.by_width[width] = dict(
                new=torch.full((s,), width, dtype=torch.int32, device=dev), slots=i32(s * width), positions=i32(s * width),
                q=q, o=torch.empty_like(q),
                workspace=torch.empty(gdn_attn_workspace_size(q, self.caches[0][0], s), dtype=torch.uint8, device=dev))

    def step(self, ids: torch.Tensor, width: int) -> torch.Tensor:
        """`width` new tokens per request (ids: [requests * width]); the logits of the last one of each."""
        m, cfg, s, b = self.model, self.model.cfg, self.requests, self.by_width[width]
        gdn_kv_plan(self.ctx, b["new"], self.owned, self.free, self.n_free, self.table, cfg.page, self.n_pages,
                    self.kv_lens, self.owned_out, self.n_free_out, self.start, b["slots"], b["positions"])
        x = m.embed[ids]
        for i in range(cfg.blocks):
            for j in range(i * cfg.gdn_per_block, (i + 1) * cfg.gdn_per_block):
                x = x + self._gdn(m.gdn[j], self.states[j], _norm(x), width)
            x = x + self._attn(m.attn[i], self.caches[i], _norm(x), b)
        # the next step starts where this one ended
        self.ctx.copy_(self.kv_lens)
        self.owned.copy_(self.owned_out)
        self.n_free.copy_(self.n_free_out)
        return _norm(x.view(s, width, -1)[:, -1]) @ m.head

    def _gdn(self, w, state, x, width):
        cfg, s = self.model.cfg, self.requests
        d, nk, nv = cfg.gdn_dim, cfg.gdn_k_heads, cfg.gdn_v_heads
        qkv = (x @ w["qkv"]).view(-1, 2 * nk + nv, d)
        q, k, v = qkv.split([nk, nk, nv], 1)
        q, k = (torch.nn.functional.normalize(t, dim=-1).contiguous() for t in (q, k))
        gates = x @ w["gates"]
        g, beta = torch.nn.functional.softplus(gates[:, :nv]).contiguous(), gates[:, nv:].sigmoid().contiguous()
        y = torch.empty(x.shape[0], nv, d, device=x.device)
        p = pack_params(d, d, nk, nv, width, s, q_scale=1.0 / math.sqrt(d))
        gdn_forward(q, k, v.contiguous(), g, beta, state, y, state, p)
        return y.view(x.shape[0], -1) @ w["out"]

    def _attn(self, w, cache, x, b):
        cfg = self.model.cfg
        d, nq, nkv = cfg.head_dim, cfg.q_heads, cfg.kv_heads
        qkv = x @ w["qkv"]
        q, k, v = (t.unflatten(1, (-1, d)) for t in qkv.split([nq * d, nkv * d, nkv * d], 1))
        gdn_rope_store(q, k, v, b["positions"], self.model.table, b["slots"], *cache, b["q"])
        gdn_attn_paged(b["q"], *cache, self.table, self.kv_lens, self.start, b["o"], b["workspace"])
        return b["o"].view(x.shape[0], -1) @ w["out"]


def _norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def generate(model: Model, prompts: torch.Tensor, steps: int):
    """Greedy tokens after `prompts` [requests, prompt] and the last step's logits: one step for the
    prompts, then `steps` decode steps as replays of one captured step."""
    s, prompt = prompts.shape
    server = Server(model, s, prompt, prompt + steps)
    logits = server.step(prompts.reshape(-1), prompt).clone()
    ids = logits.argmax(-1)
    out = [ids.clone()]

    def decode():
        logits.copy_(server.step(ids, 1))
        ids.copy_(logits.argmax(-1))

    graph = None
    for i in range(steps):
        if i == 0:  # the first decode step runs as it is: it loads what a capture must not
            decode()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    decode()
            graph.replay()
        out.append(ids.clone())
    return torch.stack(out, 1), logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--check", action="store_true", help="compare the last logits with those of one pass over all tokens")
    a = ap.parse_args(argv)
    model = Model(Config())
    prompts = torch.randint(0, model.cfg.vocab, (a.requests, a.prompt), generator=torch.Generator().manual_seed(1)).cuda()
    generate(model, prompts, min(a.steps, 3))  # warm-up
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    tokens, logits = generate(model, prompts, a.steps)
    end.record()
    torch.cuda.synchronize()
    from ._native import gdn_device_status
    print(f"{a.requests} requests, prompt {a.prompt}, {a.steps} steps: {begin.elapsed_time(end):.2f} ms, "
          f"device status {gdn_device_status()}")
    print("first request:", tokens[0, :16].tolist())
    if a.check:
        whole = torch.cat([prompts, tokens[:, :-1]], 1)  # every token that the last step has seen
        ref = Server(model, a.requests, whole.shape[1], whole.shape[1]).step(whole.reshape(-1), whole.shape[1])
        err = float((logits - ref).norm() / ref.norm())
        print(f"last logits against one pass over all {whole.shape[1]} tokens: rel-L2 {err:.2e}")
        return err
    return 0.0


if __name__ == "__main__":
    main()
