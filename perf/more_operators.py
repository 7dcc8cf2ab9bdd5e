"""Operators of a serving step with an 8-bit cache and drafted trees, as cases: plain forms, and the framework's calls.

    rope    rotary positions of queries and keys
    store   keys and values into the paged cache, rotated and quantised on the way, and the cache read back
    read    cached positions back as 16-bit keys and values
    attn    attention of the new tokens over an 8-bit paged cache
    tree    attention of a tree of drafted tokens over a paged cache of 16 or 8 bits

``run`` is the plain form (elementary torch operations in 32 bits, angles in 64)
where ``own`` is false, and the framework's calls where it is true.  ``exact``
computes the floating outputs in 64 bits.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}
TOP = {"int8": 127.0, "e4m3": 448.0}   # the largest code
DEV = "cuda"


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # queries and keys of one decode step, cut out of the fused projection's output
        dict(name="rope_decode_64", op="rope", tokens=64, heads=40, dim=128, rotary=128, interleaved=False, far=8448,
             scaling="none", dtype="bf16"),
        # a prefill step of prompts in a context stretched eightfold, half of each head rotated
        dict(name="rope_prefill_16k", op="rope", tokens=16301, heads=40, dim=128, rotary=64, interleaved=True, far=131072,
             scaling="ramp", dtype="bf16"),
        # one decode step's queries, keys and values: rotated and into an 8-bit cache
        dict(name="store_decode_64", op="store", tokens=64, pad=64, heads=32, kv_heads=8, dim=128, rotary=128,
             interleaved=False, far=8448, page=16, code="int8", dtype="bf16"),
        # a prefill step's keys and values into an 8-bit floating cache, an odd number of tokens
        dict(name="store_prefill_16k", op="store", tokens=16301, pad=256, heads=0, kv_heads=8, dim=128, rotary=0,
             interleaved=False, far=8448, page=64, code="e4m3", dtype="bf16"),
        # a short prompt's cache handed to a 16-bit consumer
        dict(name="read_300", op="read", tokens=300, kv_heads=8, dim=128, page=16, code="e4m3", dtype="fp16"),
        # the cached prefixes of a whole batch, in 16 bits
        dict(name="read_32k", op="read", tokens=32768, kv_heads=8, dim=128, page=64, code="int8", dtype="bf16"),
        # one user's decode step in a medium conversation: the smallest call, where latency counts
        dict(name="attn8_decode_1", op="attn", requests=1, mode="decode", new=1, past=2303, heads=32, kv_heads=8, dim=128,
             page=16, window=0, code="e4m3", dtype="bf16"),
        # a decode step of a batch whose contexts run from short to long
        dict(name="attn8_decode_64", op="attn", requests=64, mode="decode", new=1, past=8447, heads=32, kv_heads=8,
             dim=128, page=16, window=0, code="int8", dtype="bf16"),
        # a 2048-token chunk of a long prompt over what the cache holds already
        dict(name="attn8_chunk_2048", op="attn", requests=1, mode="even", new=2048, past=6400, heads=32, kv_heads=8,
             dim=128, page=64, window=0, code="int8", dtype="bf16"),
        # one user's small tree of drafted tokens
        dict(name="tree_1x13", op="tree", requests=1, mode="even", new=13, past=2303, heads=32, kv_heads=8, dim=128,
             page=16, window=0, code="none", dtype="bf16"),
        # a batch of trees of 64 nodes
        dict(name="tree_16x64", op="tree", requests=16, mode="even", new=64, past=4080, heads=32, kv_heads=8, dim=128,
             page=32, window=0, code="none", dtype="bf16"),
        # trees over an 8-bit cache under a sliding window, narrow heads, an odd group
        dict(name="tree_24x50_window", op="tree", requests=24, mode="mixed", new=50, past=3800, heads=28, kv_heads=4,
             dim=64, page=16, window=1024, code="int8", dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "store", "read", "attn", "attn", "tree", "tree"])
    dtype, page, dim = rng.choice(["bf16", "fp16"]), rng.choice([16, 32, 64, 128]), rng.choice([64, 128])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "rope":
        dim = rng.choice([64, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 8192), heads=rng.choice([1, 5, 12, 20, 40]), dim=dim,
                    rotary=rng.choice([dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    far=_log(rng, 512, 131072), scaling=rng.choice(["none", "linear", "ramp"]), dtype=dtype)
    if op == "store":
        turned = rng.random() < 0.7
        return dict(op=op, tokens=_log(rng, 1, 8192), pad=rng.choice([1, 64, 256]),
                    heads=kv_heads * rng.choice([1, 3, 4]) if turned else 0, kv_heads=kv_heads, dim=dim,
                    rotary=rng.choice([dim, dim // 2]) if turned else 0, interleaved=rng.random() < 0.5,
                    far=_log(rng, 512, 131072), page=page, code=rng.choice(["int8", "e4m3", "none"]) if turned else
                    rng.choice(["int8", "e4m3"]), dtype=dtype)
    if op == "read":
        return dict(op=op, tokens=_log(rng, 1, 32768), kv_heads=kv_heads, dim=dim, page=page,
                    code=rng.choice(["int8", "e4m3", "none"]), dtype=dtype)
    kv_heads = rng.choice([2, 4, 8])
    heads = kv_heads * rng.choice([1, 3, 4, 7, 8] if kv_heads < 8 else [1, 3, 4])
    past = _log(rng, 64, 8000)
    case = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, past=past, window=rng.choice([0, 0, 1024]),
                dtype=dtype)
    if op == "tree":
        requests = _log(rng, 1, 16)
        new = min(_log(rng, 2, 200), max(2, (2048 * 6400) // (requests * (past + 200))))
        return dict(case, requests=requests, mode=rng.choice(["even", "mixed"]), new=new,
                    code=rng.choice(["none", "int8", "e4m3"]))
    mode = rng.choice(["decode", "even", "mixed"])
    if mode == "decode":
        requests, new = _log(rng, 1, 64), 1
    elif mode == "even":
        requests = _log(rng, 1, 16)
        new = min(_log(rng, 2, 2048), max(2, (2048 * 8448) // (requests * (past + 2048))))
    else:
        requests = _log(rng, 2, 24)
        new = min(_log(rng, 2, 512), max(2, (2048 * 8448) // (requests * (past + 512))))
    return dict(case, requests=requests, mode=mode, new=new, code=rng.choice(["int8", "e4m3"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Host lists (cached tokens, new tokens) of the requests: fixed by the case, so that its work is."""
    g = torch.Generator().manual_seed(0x5EED)
    B, most = case["requests"], case["new"]
    past = (case["past"] * (0.02 + 0.98 * torch.rand(B, generator=g))).to(torch.int64).clamp_(min=1)
    past[-1] = case["past"]
    if case["mode"] == "mixed":   # trees of all sizes; prompt chunks beside decoding requests
        some = (2 + (most - 2) * torch.rand(B, generator=g)).to(torch.int64)
        some[0] = most
        chunk = torch.rand(B, generator=g) < (0.75 if case["op"] == "tree" else 0.25)
        chunk[0] = True
        return past, torch.where(chunk, some, 1)
    if case["mode"] == "even":
        past = torch.full((B,), case["past"], dtype=torch.int64) - torch.arange(B) * 7 % max(1, case["past"] // 2)
    return past, torch.full((B,), most, dtype=torch.int64)


def _i32(t):
    return t.to(torch.int32).to(DEV)


def _codes(code, dtype, shape, gd):
    """A cache's contents, normally distributed values, and the scales of its rows."""
    x = torch.randn(shape, generator=gd, device=DEV)
    if code == "none":
        return x.to(TYPES[dtype]), None
    scale = (0.5 + torch.rand(shape[:-1], generator=gd, device=DEV)) * 2.7 / TOP[code]
    x *= TOP[code] / 2.7
    if code == "int8":
        x.round_()
    return x.clamp_(-TOP[code], TOP[code]).to(TYPES[code]), scale


def _frequencies(rotary, scaling, base=10000.0, factor=8.0, first=4096):
    """Radians per position of each pair, in 64 bits, and the magnitude that goes with them."""
    i = torch.arange(rotary // 2, dtype=torch.float64)
    f = base ** (-2 * i / rotary)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ramp":   # pairs of few turns in the first context are stretched, pairs of many kept
        at = lambda turns: rotary * math.log(first / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rotary // 2 - 1)
        stretched = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return f * (1 - stretched) + f / factor * stretched, 0.1 * math.log(factor) + 1
    return f, 1.0


def _trees(new, words, g):
    """A random tree a request, parents before children: row t holds the bits of the nodes on the path to t's own."""
    rows = []
    for n in new.tolist():
        seen = torch.zeros((n, words * 32), dtype=torch.bool)
        parent = (torch.arange(n) - 1 - (torch.rand(n, generator=g) ** 2 * 6).to(torch.int64)).clamp(min=-1)
        for i, up in enumerate(parent.tolist()):
            if up >= 0:
                seen[i] = seen[up]
            seen[i, i] = True
        rows.append(seen)
    bits = torch.cat(rows).view(-1, words, 32).to(torch.int64) << torch.arange(32)
    return bits.sum(-1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)
    op, dt, st = case["op"], TYPES[case["dtype"]], dict(case)
    if op in ("rope", "store"):
        T, D = case["tokens"], case["dim"]
        Tp = T if op == "rope" else -(-T // case["pad"]) * case["pad"]
        # runs of positions, as prompts have them (single positions in a small step)
        start = torch.randint(0, case["far"], (Tp,), generator=g)
        run = 1 if T <= 256 else 1000
        at = torch.arange(Tp)
        positions = (start[at // run] + at % run).clamp_(max=case["far"] - 1)
        positions[T:] = -1
        st["positions"] = _i32(positions)
        f, st["magnitude"] = _frequencies(case["rotary"] or 2, case.get("scaling", "none"))
        st["frequencies"] = f.to(DEV)
    if op == "rope":
        # queries and keys are the first heads of the fused projection's rows
        H = case["heads"]
        qkv = torch.randn((T, H + 8, D), generator=gd, device=DEV).to(dt)
        st.update(x=qkv[:, :H], out=torch.empty((T, H, D), dtype=dt, device=DEV))
        return st
    if op == "store":
        H, Hk, page = case["heads"], case["kv_heads"], case["page"]
        pages = -(-(T + 512) // page)
        qkv = torch.randn((Tp, H + 2 * Hk, D), generator=gd, device=DEV).to(dt)
        st["q"], st["k"], st["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
        slots = torch.full((Tp,), -1, dtype=torch.int64)
        if T <= 256:  # decode: every token in a page of its own request
            slots[:T] = torch.randperm(pages * page, generator=g)[:T]
        else:         # prompts: runs of whole pages, in random order
            t = torch.arange(T)
            slots[:T] = torch.randperm(pages, generator=g)[t // page] * page + t % page
        st["slots"] = _i32(slots)
        for n in ("k", "v"):
            st[n + "_cache"], st[n + "_scale"] = _codes(case["code"], case["dtype"], (pages, Hk, page, D), gd)
            st[n + "_back"] = torch.empty((pages * page, Hk, D), dtype=dt, device=DEV)
        st.update(everything=torch.arange(pages * page, dtype=torch.int32, device=DEV), pages=pages,
                  q_out=torch.zeros((Tp, H, D), dtype=dt, device=DEV))
        return st
    if op == "read":
        T, Hk, page, D = case["tokens"], case["kv_heads"], case["page"], case["dim"]
        pages = -(-T // page) + 64
        for n in ("k", "v"):
            st[n + "_cache"], st[n + "_scale"] = _codes(case["code"], case["dtype"], (pages, Hk, page, D), gd)
            st[n + "_back"] = torch.empty((T, Hk, D), dtype=dt, device=DEV)
        t = torch.arange(T)
        st["slots"] = _i32(torch.randperm(pages, generator=g)[t // page] * page + t % page)
        return st
    page, H, Hk, D = case["page"], case["heads"], case["kv_heads"], case["dim"]
    past, new = _lengths(case)
    kv, total = past + new, int(new.sum())
    held = (kv + page - 1) // page
    pages, columns = int(held.sum()) + 64, int(held.max()) + 3
    order, col = torch.randperm(pages, generator=g), torch.arange(columns)
    at = ((torch.cumsum(held, 0) - held)[:, None] + col[None]).clamp_(max=pages - 1)
    st["table"] = _i32(torch.where(col[None] < held[:, None], order[at], -1))
    st["q"] = torch.randn((total, H, D), generator=gd, device=DEV).to(dt)
    for n in ("k", "v"):
        st[n + "_cache"], st[n + "_scale"] = _codes(case["code"], case["dtype"], (pages, Hk, page, D), gd)
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)])
    st.update(q_start=_i32(q_start), kv_len=_i32(kv), max_q=int(new.max()), max_kv=int(kv.max()),
              out=torch.empty((total, H, D), dtype=dt, device=DEV),
              lse=torch.empty((total, H), dtype=torch.float32, device=DEV),
              tree=_trees(new, -(-int(new.max()) // 32), g).to(DEV) if op == "tree" else None)
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"rope": _rope, "store": _store, "read": _read, "attn": _attn, "tree": _attn}[st["op"]](st)


def _own(st):
    import int4_weight_only_gemm_gb300 as w
    op = st["op"]
    if op == "rope":
        return w.w4a16_rope(st["x"], st["positions"], st["frequencies"], interleaved=st["interleaved"],
                            magnitude=st["magnitude"], out=st["out"])
    if op == "store":
        if st["rotary"]:
            w.w4a16_rope_kv_write(st["q"], st["k"], st["v"], st["positions"], st["frequencies"], st["slots"],
                                  st["k_cache"], st["v_cache"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                  interleaved=st["interleaved"], magnitude=st["magnitude"], q_out=st["q_out"])
        else:
            w.w4a16_kv_write(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"], k_scale=st["k_scale"],
                             v_scale=st["v_scale"])
        # what an 8-bit cache holds is handed on as the values it stands for
        w.w4a16_kv_read(st["k_cache"], st["v_cache"], st["everything"], st["k_back"], st["v_back"],
                        k_scale=st["k_scale"], v_scale=st["v_scale"])
        return st["q_out"], st["k_back"], st["v_back"], st["k_scale"], st["v_scale"]
    if op == "read":
        w.w4a16_kv_read(st["k_cache"], st["v_cache"], st["slots"], st["k_back"], st["v_back"], k_scale=st["k_scale"],
                        v_scale=st["v_scale"])
        return st["k_back"], st["v_back"]
    w.w4a16_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["q_start"], st["kv_len"], st["max_q"],
                            window=st["window"], out=st["out"], lse=st["lse"], k_scale=st["k_scale"],
                            v_scale=st["v_scale"], tree=st["tree"])
    return st["out"], st["lse"]


def _turned(x, st):
    """x [T, heads, d] in 32 bits with its first columns rotated; angles in 64."""
    r, half = st["rotary"], st["rotary"] // 2
    angle = st["positions"].double()[:, None, None] * st["frequencies"]
    cos, sin = (angle.cos() * st["magnitude"]).float(), (angle.sin() * st["magnitude"]).float()
    y = x.clone()
    if st["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y[..., 0:r:2], y[..., 1:r:2] = a * cos - b * sin, a * sin + b * cos
    else:
        a, b = x[..., :half], x[..., half:r]
        y[..., :half], y[..., half:r] = a * cos - b * sin, a * sin + b * cos
    return y


def _rope(st):
    return _turned(st["x"].float(), st).to(st["x"].dtype)


def _values(st, name):
    """A cache in 32 bits."""
    x = st[name + "_cache"].float()
    return x if st[name + "_scale"] is None else x * st[name + "_scale"][..., None]


def _store(st):
    T, page, code = st["tokens"], st["page"], st["code"]
    s = st["slots"][:T]
    back = []
    if st["rotary"]:
        st["q_out"][:T] = _turned(st["q"].float(), st)[:T].to(st["q"].dtype)
    for n in ("k", "v"):
        x = st[n].float()
        if st["rotary"] and n == "k":
            x = _turned(x, st)
        x = x[:T]
        if code == "none":
            st[n + "_cache"][s // page, :, s % page] = x.to(st[n].dtype)
        else:
            amax = x.abs().amax(-1)
            top = torch.full_like(amax, TOP[code])
            y = x * torch.where(amax > 0, top / amax, 0.0)[..., None]
            y = y.round() if code == "int8" else y
            st[n + "_cache"][s // page, :, s % page] = y.to(TYPES[code])
            st[n + "_scale"][s // page, :, s % page] = amax / top
        back.append(_values(st, n).transpose(1, 2).reshape(st["pages"] * page, st["kv_heads"], -1).to(st[n].dtype))
    return st["q_out"], back[0], back[1], st["k_scale"], st["v_scale"]


def _read(st):
    s, page = st["slots"], st["page"]
    return tuple(_values(st, n)[s // page, :, s % page].to(TYPES[st["dtype"]]) for n in ("k", "v"))


def _attn(st):
    q, table, q_start, kv_len, page = st["q"], st["table"], st["q_start"], st["kv_len"], st["page"]
    T, H, D = q.shape
    Hk, tree = st["kv_heads"], st["tree"]
    G, B, M, S = H // Hk, table.shape[0], st["max_q"], st["max_kv"]
    new = q_start[1:] - q_start[:-1]
    past = (kv_len - new)[:, None, None]
    i, j = torch.arange(M, device=DEV), torch.arange(S, device=DEV)
    rows = (q_start[:-1, None] + i[None]).clamp(max=T - 1)
    qp = q[rows].float().view(B, M, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, M * G, D)
    pages = table[:, :-(-S // page)].clamp(min=0)

    def cached(n):
        c = st[n + "_cache"][pages].float()
        if st[n + "_scale"] is not None:
            c = c * st[n + "_scale"][pages][..., None]
        return c.permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)[:, :, :S]

    s = torch.matmul(qp, cached("k").transpose(2, 3)) * (1.0 / math.sqrt(D))
    if tree is None:
        last = past + i[None, :, None]
        seen = j <= last
    else:   # the context, and the nodes on the path; a node's place is behind the context by its depth
        words = tree[rows]
        bit = (words[..., None] >> torch.arange(32, device=DEV)) & 1
        bit = torch.where(i[None, :, None] < new[:, None, None], bit.reshape(B, M, -1), 0)
        last = past - 1 + bit.sum(-1, keepdim=True)
        at = (j - past).clamp(0, bit.shape[-1] - 1).expand(B, M, S)
        node = (j >= past) & (j < kv_len[:, None, None]) & (torch.gather(bit, 2, at) > 0)
        seen = (j < past) | node
    if st["window"]:
        near = j > last - st["window"]
        seen = seen & near if tree is None else (seen & near) | node
    seen = seen[:, None, :, None, :]
    s = torch.where(seen, s.view(B, Hk, M, G, S), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, M * G, S), cached("v")).view(B, Hk, M, G, D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + torch.log(l)).squeeze(-1)
    t = torch.arange(T, dtype=torch.int32, device=DEV)
    r = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, M, H, D)[r, (t - q_start[r]).long()]
    return o.to(q.dtype), lse.permute(0, 2, 1, 3).reshape(B, M, H)[r, (t - q_start[r]).long()].contiguous()


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op, D = case["op"], case["dim"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * D * 4 + 4 * case["tokens"] + 4 * case["rotary"], "flops": 3 * n * case["rotary"]}
    size = D * 2 if case["code"] == "none" else D + 4   # of a cached key or value
    if op == "store":
        T, Hk, page = case["tokens"], case["kv_heads"], case["page"]
        Tp, slots = -(-T // case["pad"]) * case["pad"], -(-(T + 512) // page) * page
        write = 4 * T * case["heads"] * D + 2 * T * Hk * (2 * D + size) + 8 * Tp + 4 * case["rotary"]
        # the slots that the same pass wrote need no reading
        back = 2 * (slots - T) * Hk * size + 4 * slots * Hk * D + 4 * slots
        return {"bytes": write + back, "flops": 3 * T * (case["heads"] + Hk) * case["rotary"] + 8 * T * Hk * D}
    if op == "read":
        n = case["tokens"] * case["kv_heads"]
        return {"bytes": 2 * n * (size + 2 * D) + 4 * case["tokens"], "flops": 2 * n * D}
    past, new = _lengths(case)
    H, Hk, W, page = case["heads"], case["kv_heads"], case["window"], case["page"]
    if op == "tree":
        pairs = sum(n * (min(p, max(W - 1, 0)) + 1 if W else p + 1) for p, n in zip(past.tolist(), new.tolist()))
        keys = sum((min(p, max(W - 1, 0)) if W else p) + n for p, n in zip(past.tolist(), new.tolist()))
    else:
        pairs = sum(min(e, W) if W else e for p, n in zip(past.tolist(), new.tolist()) for e in range(p + 1, p + n + 1))
        keys = sum(p + n - max(0, p + 1 - W if W else 0) for p, n in zip(past.tolist(), new.tolist()))
    T = int(new.sum())
    mask = 4 * T * -(-int(new.max()) // 32) if op == "tree" else 0
    return {"bytes": 2 * keys * Hk * size + 4 * T * H * D + 4 * T * H + 4 * (keys // page) + mask,
            "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def _exact_turn(x, positions, st):
    """Pairs as complex numbers, each times e^(i position frequency)."""
    r = st["rotary"]
    x = x.double()
    pairs = x[..., :r].unflatten(-1, (r // 2, 2)) if st["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous())
    angle = positions.double()[:, None] * st["frequencies"][None]
    z = torch.view_as_real(z * torch.polar(torch.full_like(angle, st["magnitude"]), angle)[:, None])
    front = z.flatten(-2) if st["interleaved"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([front, x[..., r:]], -1)


def exact(case, seed):
    st = prepare(case, seed)
    op, page = case["op"], case["page"] if "page" in case else 0
    if op == "rope":
        return _exact_turn(st["x"], st["positions"], st)
    if op == "read":
        res = []
        for n in ("k", "v"):
            c = st[n + "_cache"].double()
            c = c if st[n + "_scale"] is None else c * st[n + "_scale"].double()[..., None]
            res.append(c.permute(0, 2, 1, 3).flatten(0, 1)[st["slots"].long()])
        return tuple(res)
    if op == "store":
        T = case["tokens"]
        slots = st["slots"][:T].long()
        q = st["q_out"].double()
        if case["rotary"]:
            q[:T] = _exact_turn(st["q"][:T], st["positions"][:T], st)
        res, scales = [], []
        for n in ("k", "v"):
            c = st[n + "_cache"].double()
            scale = st[n + "_scale"]
            x = st[n][:T].double()
            if case["rotary"] and n == "k":
                x = _exact_turn(x, st["positions"][:T], st)
            if scale is None:
                c = c.permute(0, 2, 1, 3).flatten(0, 1)
                c[slots] = x
                scales.append(None)
            else:
                scale = scale.double().permute(0, 2, 1).flatten(0, 1)
                c = c.permute(0, 2, 1, 3).flatten(0, 1) * scale[..., None]
                amax = x.abs().amax(-1)
                scale[slots] = amax / TOP[case["code"]]
                # which code a value next to a border gets is a decision of 32 bits: without a rotation, the values
                # that the codes stand for are exact here; with one, they have no value of their own
                y = x.float() * (TOP[case["code"]] / amax.float().double()).float()[..., None]
                y = y.round() if case["code"] == "int8" else y.to(torch.float8_e4m3fn)
                c[slots] = y.double() * scale[slots][..., None]
                scales.append(scale.unflatten(0, (st["pages"], page)).transpose(1, 2))
                if case["rotary"] and n == "k":
                    c = None
            res.append(c)
        return q, res[0], res[1], scales[0], scales[1]
    return _exact_attn(case, st)


def _exact_attn(case, st):
    """One request and key head at a time: scores, softmax and sum of the values it sees, in 64 bits."""
    q, page, Hk, W = st["q"], case["page"], case["kv_heads"], case["window"]
    G, D = case["heads"] // Hk, case["dim"]
    starts, lens = st["q_start"].tolist(), st["kv_len"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        new, pos = hi - lo, torch.arange(n, device=DEV)
        past = n - new
        page_of, slot_of = st["table"][b].long()[pos // page], pos % page
        if st["tree"] is None:
            end = torch.arange(past, n, device=DEV)
            seen = pos[None] <= end[:, None]
            if W:
                seen &= pos[None] > end[:, None] - W
        else:
            words = st["tree"][lo:hi].long() & 0xFFFFFFFF
            path = torch.stack([(words[:, k // 32] >> (k % 32)) & 1 for k in range(new)], 1).bool()
            end = past - 1 + path.sum(1)
            seen = torch.cat([(pos[None, :past] > end[:, None] - W) if W else torch.ones((new, past), dtype=torch.bool, device=DEV),
                              path], 1)
        for h in range(Hk):
            k, v = (st[c + "_cache"][page_of, h, slot_of].double() *
                    (1.0 if st[c + "_scale"] is None else st[c + "_scale"][page_of, h, slot_of].double()[:, None])
                    for c in ("k", "v"))
            a = q[lo:hi, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,jd->tgj", a, k) / math.sqrt(D)
            s.masked_fill_(~seen[:, None], -math.inf)
            out[lo:hi, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", torch.softmax(s, -1), v)
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
    return out, lse
