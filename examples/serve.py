"""Continuous batching on the GPU kernels: a small decoder with 4-bit weights
answers prompts of different lengths from a paged cache.

    python examples/serve.py [--requests 6] [--new 24] [--seed 0] [--cache bf16|int8|e4m3]

Each step takes any mixture of prompts, prompt chunks and single tokens:

    w4a16_page_plan         pages, slots and positions of the step's tokens
    per layer
        w4a16_gemm          the fused q / k / v projection
        w4a16_rope_kv_write rotary positions, the new keys and values into the cache
        w4a16_paged_attention
        w4a16_gemm          output projection
        w4a16_gemm_gate_up_silu, w4a16_gemm    the MLP
    w4a16_gemm              the vocabulary head, for every request's last token
    w4a16_sample            temperature, top-k, top-p and min-p per request

`Server.verify` takes a tree of drafted tokens a request instead: one step gives
the logits behind every node, the longest path that the model agrees with is
kept, and its keys and values move to the places behind each other
(w4a16_kv_read, w4a16_kv_write).  Norms are plain PyTorch, the weights random.
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
    cache: str = "bf16"      # or "int8", "e4m3"


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


class Cache:
    """Keys and values of a layer."""

    def __init__(self, cfg: Config):
        shape = (cfg.pages, cfg.kv_heads, cfg.page_size, cfg.head_dim)
        dtype = {"bf16": torch.bfloat16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}[cfg.cache]
        self.pages = [torch.zeros(shape, dtype=torch.int8 if dtype.itemsize == 1 else dtype, device="cuda").view(dtype)
                      for _ in range(2)]
        self.scales = {} if cfg.cache == "bf16" else {
            n: torch.zeros(shape[:3], device="cuda") for n in ("k_scale", "v_scale")}

    def move(self, source, target):
        """Keys and values from the slots `source` to the slots `target`, as they are: of an 8-bit cache two codes at a time,
        as 16-bit numbers that are copied bit for bit, and the scales."""
        pages = [c.view(torch.bfloat16) for c in self.pages]
        _, heads, size, d = pages[0].shape
        k, v = torch.empty(2, source.numel(), heads, d, dtype=torch.bfloat16, device="cuda")
        w.w4a16_kv_read(*pages, source, k, v)
        w.w4a16_kv_write(k, v, target, *pages)
        source, target = source.long(), target.long()
        for s in self.scales.values():
            s[target // size, :, target % size] = s[source // size, :, source % size]


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
        self.caches = [Cache(c) for _ in range(c.layers)]
        self.frequencies, _ = w.w4a16_rope_frequencies(c.head_dim)

    def __call__(self, tokens, plan, table, max_q, tree=None):
        """Logits [B, vocab] behind every request's last token; tokens [T] in request order.  With a tree, (mask [T,
        words], positions [T]) of the tokens as its nodes: logits [T, vocab] behind every node."""
        c = self.cfg
        q_start, kv_len, positions, slots, _ = plan
        mask = None
        if tree is not None:
            mask, positions = tree
        x = self.embed[tokens.long()]
        T = x.shape[0]
        for (qkv, o_proj, gate_up, down), cache in zip(self.blocks, self.caches):
            q, k, v = qkv(norm(x)).view(T, -1, c.head_dim).split([c.heads, c.kv_heads, c.kv_heads], dim=1)
            w.w4a16_rope_kv_write(q, k, v, positions, self.frequencies, slots, *cache.pages, q_out=q, **cache.scales)
            a = w.w4a16_paged_attention(q, *cache.pages, table, q_start, kv_len, max_q, window=c.window, tree=mask,
                                        **cache.scales)
            x = x + o_proj(a.view(T, -1))
            x = x + down(gate_up(norm(x)))
        return self.head(norm(x if tree is not None else x[q_start[1:].long() - 1]))


def _starts(counts):
    return [sum(counts[:i]) for i in range(len(counts))]


class Server:
    """Requests with a row of the block table each; pages go back when a request is done."""

    def __init__(self, model: Model, requests: int):
        c = self.cfg = model.cfg
        self.model = model
        self.table = torch.full((requests, c.max_pages), -1, dtype=torch.int32, device="cuda")
        self.free = list(range(c.pages))
        self.past = [0] * requests

    def _plan(self, new):
        """Pages, slots and positions of so many new tokens a request; what it needs of `free` is gone then."""
        c = self.cfg
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
        return plan

    def step(self, tokens):
        """Takes each request's new tokens (lists, none empty) and gives the logits behind them."""
        new = [len(t) for t in tokens]
        plan = self._plan(new)
        self.past = [p + n for p, n in zip(self.past, new)]
        tokens = torch.tensor([t for row in tokens for t in row], dtype=torch.int32, device="cuda")
        return self.model(tokens, plan, self.table, max(new))

    def verify(self, trees):
        """Takes a tree a request, a list of (parent, token) with parents before children; node 0, parent -1, is the
        request's last token, which is not in the cache yet, the others are drafts.  Gives each request's next tokens
        (the drafts on the longest path that the model's likeliest tokens follow, and its token behind them)."""
        new = [len(t) for t in trees]
        seen = torch.zeros((sum(new), -(-max(new) // 32) * 32), dtype=torch.bool)
        depth, at = [], 0
        for n, nodes in zip(new, trees):
            for i, (parent, _) in enumerate(nodes):
                if parent >= 0:
                    seen[at + i] = seen[at + parent]
                seen[at + i, i] = True
                depth.append(depth[at + parent] + 1 if parent >= 0 else 0)
            at += n
        mask = (seen.view(at, -1, 32).long() << torch.arange(32)).sum(-1).to(torch.int32).cuda()
        ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        positions = ints([p + d for p, n, s in zip(self.past, new, _starts(new)) for d in depth[s:s + n]])
        plan = self._plan(new)
        logits = self.model(ints([t for nodes in trees for _, t in nodes]), plan, self.table, max(new), (mask, positions))
        best, out, source, target = logits.argmax(-1).tolist(), [], [], []
        for r, (nodes, s) in enumerate(zip(trees, _starts(new))):
            path = [0]
            while (child := next((i for i, (p, t) in enumerate(nodes) if p == path[-1] and t == best[s + path[-1]]), None)):
                path.append(child)
            out.append([nodes[i][1] for i in path[1:]] + [best[s + path[-1]]])
            source += [s + i for at, i in enumerate(path) if i != at]   # (the others lie in place)
            target += [s + at for at, i in enumerate(path) if i != at]
            # pages behind the path's last position go back
            up = lambda n: -(-n // self.cfg.page_size)
            held = up(self.past[r] + len(path))
            self.free += self.table[r, held:up(self.past[r] + new[r])].tolist()
            self.table[r, held:] = -1
            self.past[r] += len(path)
        slots = plan[3]
        if source:
            for cache in self.model.caches:
                cache.move(slots[ints(source).long()], slots[ints(target).long()])
        return out

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
    p.add_argument("--cache", choices=["bf16", "int8", "e4m3"], default="bf16")
    a = p.parse_args()
    model, g = Model(Config(cache=a.cache), a.seed), torch.Generator().manual_seed(a.seed)
    prompts = [torch.randint(0, model.cfg.vocab, (n,), generator=g).tolist()
               for n in torch.randint(1, 300, (a.requests,), generator=g).tolist()]
    new = [a.new - i % 3 for i in range(a.requests)]
    for i, tokens in enumerate(generate(model, prompts, new, 0.8, 50, 0.95, 0.02, a.seed)):
        print(f"request {i}: {len(prompts[i])} prompt tokens ->", *tokens[:12], "..." if len(tokens) > 12 else "")


if __name__ == "__main__":
    main()
