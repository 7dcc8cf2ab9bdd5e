"""Continuous batching on the GPU kernels: a small decoder with 4-bit weights
answers prompts of different lengths from a paged cache.

    python examples/serve.py [--requests 6] [--new 24] [--seed 0]

Each step takes any mixture of prompts, prompt chunks and single tokens:

    w4a16_page_plan         pages, slots and positions of the step's tokens
    per layer
        w4a16_gemm          the fused q / k / v projection
        w4a16_kv_write      the new keys and values into the cache
        w4a16_paged_attention
        w4a16_gemm          output projection
        w4a16_gemm_gate_up_silu, w4a16_gemm    the MLP
    w4a16_gemm              the vocabulary head, for every request's last token
    w4a16_sample            temperature, top-k, top-p and min-p per request

Norms and the rotary embedding are plain PyTorch, the weights random.
"""
from __future__ import annotations

import argparse
import sys
from dataclasses import dataclass
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
import int4_weight_only_gemm_gb300 as w  # noqa: E402


@dataclass
class Config:
    hidden: int = 1024
    mlp: int = 2048
    heads: int = 8
    kv_heads: int = 2
    head_dim: int = 128
    layers: int = 2
    vocab: int = 8192
    page_size: int = 16
    pages: int = 512
    max_pages: int = 64      # of a request
    window: int = 0


class Linear:
    """A 4-bit weight [K, N] in the device layout."""

    def __init__(self, K, N, gen, gate_up=False):
        codes = torch.randint(-2 ** 31, 2 ** 31, (K // 8, N), generator=gen, dtype=torch.int64).to(torch.int32).cuda()
        self.codes = w.w4a16_pack_gate_up(codes) if gate_up else w.w4a16_pack(codes)
        # 0 .. 15 around a zero point of 8: a standard deviation of 4.6 steps
        self.scales = torch.full((K // 128, N), 1.0 / (4.6 * K ** 0.5), dtype=torch.float16, device="cuda")
        self.zeros = torch.full((K // 128, N // 8), -0x77777778, dtype=torch.int32, device="cuda")  # 8 in every nibble
        self.gate_up = gate_up

    def __call__(self, x):
        f = w.w4a16_gemm_gate_up_silu if self.gate_up else w.w4a16_gemm
        return f(x, self.codes, self.scales, self.zeros)


def norm(x):
    return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


def rotate(x, positions):
    """Rotary embedding of [T, heads, head_dim], in place."""
    half = x.shape[-1] // 2
    angle = positions.float()[:, None] * 10000.0 ** (-torch.arange(half, device=x.device).float() / half)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    a, b = x[..., :half].float(), x[..., half:].float()
    x[..., :half], x[..., half:] = (a * cos - b * sin).to(x.dtype), (a * sin + b * cos).to(x.dtype)


class Model:
    def __init__(self, cfg: Config, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        c = self.cfg = cfg
        self.embed = torch.randn(c.vocab, c.hidden, generator=g).to(torch.bfloat16).cuda()
        wide = (c.heads + 2 * c.kv_heads) * c.head_dim
        self.blocks = [(Linear(c.hidden, wide, g), Linear(c.heads * c.head_dim, c.hidden, g),
                        Linear(c.hidden, 2 * c.mlp, g, gate_up=True), Linear(c.mlp, c.hidden, g))
                       for _ in range(c.layers)]
        self.head = Linear(c.hidden, c.vocab, g)
        shape = (c.pages, c.kv_heads, c.page_size, c.head_dim)
        self.caches = [(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"),
                        torch.zeros(shape, dtype=torch.bfloat16, device="cuda")) for _ in range(c.layers)]

    def __call__(self, tokens, plan, table, max_q):
        """Logits [B, vocab] behind every request's last token; tokens [T] in request order."""
        c = self.cfg
        q_start, kv_len, positions, slots, _ = plan
        x = self.embed[tokens.long()]
        T = x.shape[0]
        for (qkv, o_proj, gate_up, down), (k_cache, v_cache) in zip(self.blocks, self.caches):
            y = qkv(norm(x)).view(T, c.heads + 2 * c.kv_heads, c.head_dim)
            rotate(y[:, :c.heads + c.kv_heads], positions)
            q, k, v = y.split([c.heads, c.kv_heads, c.kv_heads], dim=1)
            w.w4a16_kv_write(k, v, slots, k_cache, v_cache)
            a = w.w4a16_paged_attention(q, k_cache, v_cache, table, q_start, kv_len, max_q, window=c.window)
            x = x + o_proj(a.view(T, -1))
            x = x + down(gate_up(norm(x)))
        return self.head(norm(x[q_start[1:].long() - 1]))


class Server:
    """Requests with a row of the block table each; pages go back when a request is done."""

    def __init__(self, model: Model, requests: int):
        c = self.cfg = model.cfg
        self.model = model
        self.table = torch.full((requests, c.max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = list(range(c.pages))
        self.past = [0] * requests

    def step(self, tokens):
        """Takes each request's new tokens (lists, none empty) and gives the logits behind them."""
        c = self.cfg
        new = [len(t) for t in tokens]
        up = lambda n: -(-n // c.page_size)
        pages = sum(up(p + n) - up(p) for p, n in zip(self.past, new))
        if pages > len(self.free):
            raise RuntimeError("the cache is full")
        if max(up(p + n) for p, n in zip(self.past, new)) > c.max_pages:
            raise RuntimeError("a request is longer than its row of the block table")
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        plan = w.w4a16_page_plan(ints(self.past), ints(new), ints(self.free), self.table, c.page_size,
                                 max_tokens=sum(new))
        del self.free[:pages]
        self.past = [p + n for p, n in zip(self.past, new)]
        return self.model(ints([t for row in tokens for t in row]), plan, self.table, max(new))

    def drop(self, keep):
        """Keeps the requests of these indices."""
        for r in set(range(len(self.past))) - set(keep):
            self.free += self.table[r, :-(-self.past[r] // self.cfg.page_size)].tolist()
        self.table = self.table[keep].contiguous()
        self.past = [self.past[r] for r in keep]


def generate(model, prompts, new, temperature=0.0, top_k=0, top_p=1.0, min_p=0.0, seed=0):
    """The prompts' continuations; prompt i stops after new[i] tokens.  temperature 0: the likeliest token."""
    server, gen = Server(model, len(prompts)), torch.Generator("cuda").manual_seed(seed)
    out, live, feed = [[] for _ in prompts], list(range(len(prompts))), [list(p) for p in prompts]
    while live:
        logits = server.step(feed)
        B = len(live)
        ones = torch.ones(B, device="cuda")
        noise = torch.empty(logits.shape, device="cuda").exponential_(generator=gen)
        token = w.w4a16_sample(logits, noise, ones * temperature,
                               torch.full((B,), top_k, dtype=torch.int32, device="cuda"), ones * top_p, ones * min_p)
        for r, t in zip(live, token.tolist()):
            out[r].append(t)
        stay = [i for i, r in enumerate(live) if len(out[r]) < new[r]]
        if len(stay) < B:
            server.drop(stay)
            live = [live[i] for i in stay]
        feed = [[out[r][-1]] for r in live]
    return out


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--requests", type=int, default=6)
    p.add_argument("--new", type=int, default=24)
    p.add_argument("--seed", type=int, default=0)
    a = p.parse_args()
    model, g = Model(Config(), a.seed), torch.Generator().manual_seed(a.seed)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist()
               for n in torch.randint(1, 300, (a.requests,), generator=g).tolist()]
    new = [a.new - i % 3 for i in range(a.requests)]
    for i, tokens in enumerate(generate(model, prompts, new, 0.8, 50, 0.95, 0.02, a.seed)):
        print(f"request {i}: {len(prompts[i])} prompt tokens ->", *tokens[:12], "..." if len(tokens) > 12 else "")


if __name__ == "__main__":
    main()
