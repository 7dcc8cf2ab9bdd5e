"""The paged-serving operators as cases: what each one computes in plain form, and the framework's call for it.

    plan    block tables, slot map and positions of a batch, built from the requests' lengths
    write   new keys and values into the paged cache
    attn    attention of the new tokens of every request over its paged cache
    sample  temperature, top-k, top-p and min-p sampling from given random numbers

``run`` is the plain form (elementary torch operations in 32 bits) where ``own``
is false, and the framework's call where it is true.  ``exact`` computes the
floating outputs in 64 bits.
"""
import math

import torch

own = False

VOCAB = 151936          # columns of the vocabulary head
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
DEV = "cuda"


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the tables of one decode step of a server with 64 requests in flight
        dict(name="plan_decode_64", op="plan", requests=64, past=8448, new=1, starts=0.0, page=16, pad=64),
        # a large scheduler step: most requests decode, an eighth of them bring a chunk of up to 2048 prompt tokens
        dict(name="plan_chunks_2048", op="plan", requests=2048, past=8192, new=2048, starts=0.125, page=16, pad=256),
        # keys and values of one decode step, cut out of the fused projection's output
        dict(name="write_decode_64", op="write", tokens=64, pad=64, kv_heads=8, dim=128, page=16, dtype="bf16"),
        # a prefill step's keys and values: many prompts, an odd number of tokens
        dict(name="write_prefill_16k", op="write", tokens=16301, pad=256, kv_heads=8, dim=128, page=64, dtype="bf16"),
        # one user's decode step in a medium conversation: the smallest call, where latency counts
        dict(name="attn_decode_1", op="attn", requests=1, mode="decode", new=1, past=2303, heads=32, kv_heads=8, dim=128,
             page=16, window=0, block=False, dtype="bf16"),
        # a decode step of a batch whose contexts run from short to long
        dict(name="attn_decode_64", op="attn", requests=64, mode="decode", new=1, past=8447, heads=32, kv_heads=8,
             dim=128, page=16, window=0, block=False, dtype="bf16"),
        # batched verification of 16-token draft blocks
        dict(name="attn_verify_16", op="attn", requests=16, mode="even", new=16, past=4080, heads=32, kv_heads=8,
             dim=128, page=32, window=0, block=False, dtype="bf16"),
        # a 2048-token chunk of a long prompt over what the cache holds already
        dict(name="attn_chunk_2048", op="attn", requests=1, mode="even", new=2048, past=6400, heads=32, kv_heads=8,
             dim=128, page=64, window=0, block=False, dtype="bf16"),
        # a mixed step with a sliding window: decoding requests beside prompt chunks, narrow heads, odd group
        dict(name="attn_mixed_window", op="attn", requests=24, mode="mixed", new=300, past=3800, heads=28, kv_heads=4,
             dim=64, page=16, window=1024, block=False, dtype="fp16"),
        # one user's next token with the usual filters
        dict(name="sample_1", op="sample", rows=1, vocab=VOCAB, filters="kp", dtype="bf16"),
        # a batch in which every request has filters of its own
        dict(name="sample_64", op="sample", rows=64, vocab=VOCAB, filters="all", dtype="bf16"),
        # a large batch sampled from the whole distribution (rollouts), logits in 32 bits
        dict(name="sample_256_plain", op="sample", rows=256, vocab=VOCAB, filters="none", dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "write", "attn", "attn", "sample", "sample"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        requests, starts = _log(rng, 1, 2048), rng.choice([0.0, 0.125])
        new = min(_log(rng, 1, 2048), max(1, int(2 ** 18 / requests / (starts or 1.0))))
        return dict(op=op, requests=requests, past=_log(rng, 1, 8192), new=new, starts=starts, page=page,
                    pad=rng.choice([1, 64, 256]))
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 16384), pad=rng.choice([1, 64, 256]), kv_heads=rng.choice([1, 2, 4, 8]),
                    dim=rng.choice([64, 128]), page=page, dtype=rng.choice(["bf16", "fp16"]))
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, 256), vocab=rng.choice([_log(rng, 2000, VOCAB), VOCAB]),
                    filters=rng.choice(["none", "k", "p", "minp", "kp", "all"]), dtype=rng.choice(["bf16", "f32"]))
    mode = rng.choice(["decode", "even", "mixed"])
    kv_heads = rng.choice([2, 4, 8])
    heads = kv_heads * rng.choice([1, 3, 4, 7, 8] if kv_heads < 8 else [1, 3, 4])
    past = _log(rng, 64, 8000)
    if mode == "decode":
        requests, new = _log(rng, 1, 64), 1
    elif mode == "even":
        requests = _log(rng, 1, 16)
        new = min(_log(rng, 2, 2048), max(2, (2048 * 8448) // (requests * (past + 2048))))
    else:
        requests = _log(rng, 2, 24)
        new = min(_log(rng, 2, 512), max(2, (2048 * 8448) // (requests * (past + 512))))
    return dict(op=op, requests=requests, mode=mode, new=new, past=past, heads=heads, kv_heads=kv_heads,
                dim=rng.choice([64, 128]), page=page, window=rng.choice([0, 0, 1024]),
                block=mode == "even" and rng.random() < 0.3, dtype=rng.choice(["bf16", "fp16"]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """Host lists (cached tokens, new tokens) of the requests: fixed by the case, so that its work is."""
    g = torch.Generator().manual_seed(0x5EED)
    B = case["requests"]
    u = torch.rand(B, generator=g)
    past = (case["past"] * (0.02 + 0.98 * u)).to(torch.int64).clamp_(min=1)
    past[-1] = case["past"]
    if case["op"] == "plan":
        chunk = torch.rand(B, generator=g) < case["starts"]
        some = (1 + (case["new"] - 1) * torch.rand(B, generator=g)).to(torch.int64)
        new = torch.where(chunk, some, 1) if case["starts"] else some
        past = torch.where(chunk & (torch.rand(B, generator=g) < 0.5), 0, past)  # the prompt's first chunk
    elif case["mode"] == "mixed":
        chunk = torch.rand(B, generator=g) < 0.25
        chunk[0] = True
        some = (2 + (case["new"] - 2) * torch.rand(B, generator=g)).to(torch.int64)
        some[0] = case["new"]
        new = torch.where(chunk, some, 1)
    else:
        new = torch.full((B,), case["new"], dtype=torch.int64)
        if case["mode"] == "even":
            past = torch.full((B,), case["past"], dtype=torch.int64) - torch.arange(B) * 7 % max(1, case["past"] // 2)
    return past, new


def _i32(t):
    return t.to(torch.int32).to(DEV)


def _table(past, page, columns, pages, g):
    """Block table of the pages that hold `past` tokens, and the free pages, both in random order."""
    held = (past + page - 1) // page
    order = torch.randperm(pages, generator=g)
    start = torch.cumsum(held, 0) - held
    col = torch.arange(columns)
    at = (start[:, None] + col[None]).clamp_(max=pages - 1)
    return torch.where(col[None] < held[:, None], order[at], -1), order[int(held.sum()):]


def _sizes(case):
    """Host sizes of a plan or an attention case."""
    past, new = _lengths(case)
    page = case["page"]
    need = (past + new + page - 1) // page
    return past, new, int(need.max()), int(need.sum())


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    st = dict(case)
    if op == "plan":
        past, new, columns, pages = _sizes(case)
        columns += 3
        pages += 64
        table, free = _table(past, case["page"], columns, pages, g)
        total = int(new.sum())
        T = -(-total // case["pad"]) * case["pad"]
        B = case["requests"]
        st.update(past=_i32(past), new=_i32(new), free=_i32(free), table=_i32(table), T=T,
                  q_start=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                  kv_len=torch.empty(B, dtype=torch.int32, device=DEV),
                  positions=torch.empty(T, dtype=torch.int32, device=DEV),
                  slots=torch.empty(T, dtype=torch.int32, device=DEV),
                  used=torch.empty(1, dtype=torch.int32, device=DEV))
    elif op == "write":
        dt, T, H, D, page = TYPES[case["dtype"]], case["tokens"], case["kv_heads"], case["dim"], case["page"]
        Tp = -(-T // case["pad"]) * case["pad"]
        pages = -(-(T + 4096) // page)
        # keys and values are slices of the fused projection's output, behind 4 query heads a key head
        qkv = torch.randn((Tp, 6 * H * D), generator=gd, device=DEV).to(dt)
        st["k"] = qkv[:, 4 * H * D:5 * H * D].view(Tp, H, D)
        st["v"] = qkv[:, 5 * H * D:].view(Tp, H, D)
        slots = torch.full((Tp,), -1, dtype=torch.int64)
        if T <= 256:  # decode: every token in a page of its own request
            slots[:T] = torch.randperm(pages * page, generator=g)[:T]
        else:         # prompts: runs of whole pages, in random order
            order = torch.randperm(pages, generator=g)
            t = torch.arange(T)
            slots[:T] = order[t // page] * page + t % page
        st["slots"] = _i32(slots)
        for name in ("k_cache", "v_cache"):
            st[name] = torch.randn((pages, H, page, D), generator=gd, device=DEV).to(dt)
    elif op == "attn":
        dt, page = TYPES[case["dtype"]], case["page"]
        past, new, columns, pages = _sizes(case)
        kv = past + new
        table, _ = _table(kv, page, columns, pages, g)
        total = int(new.sum())
        H, Hk, D = case["heads"], case["kv_heads"], case["dim"]
        st["q"] = torch.randn((total, H, D), generator=gd, device=DEV).to(dt)
        for name in ("k_cache", "v_cache"):
            st[name] = torch.randn((pages, Hk, page, D), generator=gd, device=DEV).to(dt)
        q_start = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(new, 0)])
        st.update(table=_i32(table), q_start=_i32(q_start), kv_len=_i32(kv), max_q=int(new.max()),
                  max_kv=int(kv.max()), out=torch.empty((total, H, D), dtype=dt, device=DEV),
                  lse=torch.empty((total, H), dtype=torch.float32, device=DEV))
    else:
        R, V = case["rows"], case["vocab"]
        # a broad body of logits with a heavy head, as a language model gives
        x = torch.randn((R, V), generator=gd, device=DEV) * 2.2
        x += 14.0 * torch.rand((R, V), generator=gd, device=DEV) ** 64
        st["logits"] = x.to(TYPES[case["dtype"]])
        del x
        st["noise"] = torch.empty((R, V), device=DEV).exponential_(generator=gd)
        temperature = 0.6 + 0.7 * torch.rand(R, generator=g)
        temperature[torch.rand(R, generator=g) < 0.1] = 0.0  # some requests decode greedily
        f = case["filters"]
        top_k = torch.randint(5, 120, (R,), generator=g)
        top_p = 0.7 + 0.29 * torch.rand(R, generator=g)
        min_p = 0.01 + 0.1 * torch.rand(R, generator=g)
        if f == "all":  # requests with some of the filters off
            top_k[torch.rand(R, generator=g) < 0.5] = 0
            top_p[torch.rand(R, generator=g) < 0.25] = 1.0
            min_p[torch.rand(R, generator=g) < 0.5] = 0.0
        st.update(temperature=temperature.to(DEV),
                  top_k=_i32(top_k) if f in ("k", "kp", "all") else None,
                  top_p=top_p.to(DEV) if f in ("p", "kp", "all") else None,
                  min_p=min_p.to(DEV) if f in ("minp", "all") else None,
                  token=torch.empty(R, dtype=torch.int32, device=DEV),
                  logprob=torch.empty(R, dtype=torch.float32, device=DEV))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _own(st)
    return {"plan": _plan, "write": _write, "attn": _attn, "sample": _sample}[st["op"]](st)


def _own(st):
    import int4_weight_only_gemm_gb300 as w
    op = st["op"]
    if op == "plan":
        w.w4a16_page_plan(st["past"], st["new"], st["free"], st["table"], st["page"], st["q_start"], st["kv_len"],
                          st["positions"], st["slots"], st["used"])
        return st["table"], st["q_start"], st["kv_len"], st["positions"], st["slots"], st["used"]
    if op == "write":
        w.w4a16_kv_write(st["k"], st["v"], st["slots"], st["k_cache"], st["v_cache"])
        return st["k_cache"], st["v_cache"]
    if op == "attn":
        w.w4a16_paged_attention(st["q"], st["k_cache"], st["v_cache"], st["table"], st["q_start"], st["kv_len"],
                                st["max_q"], window=st["window"], block=st["block"], out=st["out"], lse=st["lse"])
        return st["out"], st["lse"]
    w.w4a16_sample(st["logits"], st["noise"], st["temperature"], st["top_k"], st["top_p"], st["min_p"],
                   token=st["token"], logprob=st["logprob"])
    return st["token"], st["logprob"]


def _plan(st):
    past, new, page = st["past"], st["new"], st["page"]
    held, need = (past + page - 1) // page, (past + new + page - 1) // page
    more = need - held
    first = torch.cumsum(more, 0) - more
    col = torch.arange(st["table"].shape[1], device=DEV)[None]
    at = first[:, None] + col - held[:, None]
    F = st["free"].numel()
    fresh = torch.where(at < F, st["free"][at.clamp(0, F - 1)], -1)
    table = torch.where(col < held[:, None], st["table"], torch.where(col < need[:, None], fresh, -1))
    q_start = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), torch.cumsum(new, 0)]).to(torch.int32)
    t = torch.arange(st["T"], dtype=torch.int32, device=DEV)
    live = t < q_start[-1]
    r = torch.searchsorted(q_start[1:].contiguous(), t, right=True).clamp(max=past.numel() - 1)
    pos = past[r] + t - q_start[r]
    entry = table[r, (pos // page).clamp(0, table.shape[1] - 1)]
    slots = torch.where(live & (entry >= 0), entry * page + pos % page, -1)
    return (table.to(torch.int32), q_start, past + new, torch.where(live, pos, -1).to(torch.int32),
            slots.to(torch.int32), more.sum().to(torch.int32).reshape(1))


def _write(st):
    n, page = st["tokens"], st["page"]
    s = st["slots"][:n]
    st["k_cache"][s // page, :, s % page] = st["k"][:n]
    st["v_cache"][s // page, :, s % page] = st["v"][:n]
    return st["k_cache"], st["v_cache"]


def _attn(st):
    q, table, q_start, kv_len, page = st["q"], st["table"], st["q_start"], st["kv_len"], st["page"]
    T, H, D = q.shape
    Hk = st["kv_heads"]
    G, B, M, S = H // Hk, table.shape[0], st["max_q"], st["max_kv"]
    new = q_start[1:] - q_start[:-1]
    i, j = torch.arange(M, device=DEV), torch.arange(S, device=DEV)
    rows = (q_start[:-1, None] + i[None]).clamp(max=T - 1)
    qp = q[rows].float().view(B, M, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hk, M * G, D)
    pages = table[:, :-(-S // page)].clamp(min=0)

    def cached(c):
        return c[pages].float().permute(0, 2, 1, 3, 4).reshape(B, Hk, -1, D)[:, :, :S]

    s = torch.matmul(qp, cached(st["k_cache"]).transpose(2, 3)) * (1.0 / math.sqrt(D))
    last = (kv_len[:, None] - 1).expand(B, M) if st["block"] else kv_len[:, None] - new[:, None] + i[None]
    seen = j <= last[..., None]
    if st["window"]:
        seen = seen & (j > last[..., None] - st["window"])
    seen = seen[:, None, :, None, :]
    s = torch.where(seen, s.view(B, Hk, M, G, S), -math.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, M * G, S), cached(st["v_cache"])).view(B, Hk, M, G, D)
    o = torch.where(l > 0, o / l, 0.0)
    lse = (m + torch.log(l)).squeeze(-1)
    t = torch.arange(T, dtype=torch.int32, device=DEV)
    r = torch.searchsorted(q_start[1:].contiguous(), t, right=True)
    o = o.permute(0, 2, 1, 3, 4).reshape(B, M, H, D)[r, (t - q_start[r]).long()]
    return o.to(q.dtype), lse.permute(0, 2, 1, 3).reshape(B, M, H)[r, (t - q_start[r]).long()].contiguous()


def _sample(st):
    x = st["logits"].float()
    R, V = x.shape
    temperature = st["temperature"][:, None]
    greedy = temperature <= 0
    z = x / torch.where(greedy, 1.0, temperature)
    logprob = z - torch.logsumexp(z, -1, keepdim=True)
    zs, order = torch.sort(z, dim=-1, descending=True, stable=True)
    rank = torch.arange(V, device=DEV)[None]
    keep = torch.ones_like(zs, dtype=torch.bool)
    if st["top_k"] is not None:
        k = st["top_k"][:, None]
        keep = (k <= 0) | (rank < k)
    if st["top_p"] is not None:
        p = torch.where(keep, torch.exp(zs - zs[:, :1]), 0.0)
        before = torch.cumsum(p, -1) - p
        top_p = st["top_p"][:, None]
        keep = keep & ((top_p >= 1) | (before < top_p * p.sum(-1, keepdim=True)) | (rank == 0))
    if st["min_p"] is not None:
        least = st["min_p"][:, None]
        keep = keep & ((least <= 0) | (zs - zs[:, :1] >= torch.log(least)) | (rank == 0))
    score = torch.where(keep, zs - torch.log(torch.gather(st["noise"], 1, order)), -math.inf)
    best = score.amax(-1, keepdim=True)
    token = torch.where(score == best, order, V).amin(-1)   # equal scores: the lowest index
    token = torch.where(greedy[:, 0], order[:, 0], token)
    return token.to(torch.int32), torch.gather(logprob, 1, token[:, None])[:, 0]


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "plan":
        past, new, columns, _ = _sizes(case)
        B, page = case["requests"], case["page"]
        held = int(((past + page - 1) // page).sum())
        need = int(((past + new + page - 1) // page).sum())
        T = -(-int(new.sum()) // case["pad"]) * case["pad"]
        # the entries of the pages held are neither read nor written, but for the one that a token's slot needs
        return {"bytes": 4 * (2 * B + (need - held) + B + (B * (columns + 3) - held) + 2 * B + 1 + 2 * T + 1), "flops": 0}
    if op == "write":
        T, size = case["tokens"], case["kv_heads"] * case["dim"] * 2
        return {"bytes": 4 * T * size + 4 * (-(-T // case["pad"]) * case["pad"]), "flops": 0}
    if op == "attn":
        past, new, columns, _ = _sizes(case)
        H, Hk, D, W = case["heads"], case["kv_heads"], case["dim"], case["window"]
        pairs = keys = 0
        for p, n in zip(past.tolist(), new.tolist()):
            ends = [p + n] * n if case["block"] else range(p + 1, p + n + 1)
            pairs += sum(min(e, W) if W else e for e in ends)
            first = max(0, (p + n if case["block"] else p + 1) - W) if W else 0
            keys += p + n - first
        T = int(new.sum())
        return {"bytes": 4 * keys * Hk * D + 4 * T * H * D + 4 * T * H + 4 * (keys // case["page"]),
                "flops": 4 * D * H * pairs}
    n = case["rows"] * case["vocab"]
    size = 2 if case["dtype"] == "bf16" else 4
    # with filters, random numbers are needed for the few tokens that are left only
    return {"bytes": n * size + (4 * n if case["filters"] == "none" else 0), "flops": 4 * n}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "plan":
        return None
    st = prepare(case, seed)
    if op == "write":
        res = []
        for x, c in ((st["k"], st["k_cache"]), (st["v"], st["v_cache"])):
            c = c.double().permute(0, 2, 1, 3).reshape(-1, case["kv_heads"], case["dim"])
            c.index_copy_(0, st["slots"][:case["tokens"]].long(), x[:case["tokens"]].double())
            res.append(c.view(-1, case["page"], case["kv_heads"], case["dim"]).permute(0, 2, 1, 3).contiguous())
        return tuple(res)
    if op == "attn":
        return _exact_attn(case, st)
    x = st["logits"].double()
    t = st["temperature"].double()
    z = x / torch.where(t > 0, t, torch.ones_like(t))[:, None]
    z -= z.amax(1, keepdim=True)
    token = _sample(st)[0].long()  # the drawn token is a whole number; its log-probability is what is computed
    return None, z.gather(1, token[:, None])[:, 0] - z.exp().sum(1).log()


def _exact_attn(case, st):
    """One request and key head at a time: scores, softmax and sum of the values it sees, in 64 bits."""
    q, page, Hk = st["q"], case["page"], case["kv_heads"]
    G, D = case["heads"] // Hk, case["dim"]
    starts, lens = st["q_start"].tolist(), st["kv_len"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=DEV)
    for b, n in enumerate(lens):
        lo, hi = starts[b], starts[b + 1]
        pos = torch.arange(n, device=DEV)
        page_of, slot_of = st["table"][b].long()[pos // page], pos % page
        for h in range(Hk):
            k, v = (st[c][page_of, h, slot_of].double() for c in ("k_cache", "v_cache"))
            a = q[lo:hi, h * G:(h + 1) * G].double()
            s = torch.einsum("tgd,jd->tgj", a, k) / math.sqrt(D)
            end = torch.full((hi - lo,), n - 1, device=DEV) if case["block"] else torch.arange(n - (hi - lo), n, device=DEV)
            hidden = pos[None] > end[:, None]
            if case["window"]:
                hidden |= pos[None] <= end[:, None] - case["window"]
            s.masked_fill_(hidden[:, None], -math.inf)
            w = torch.softmax(s, -1)
            out[lo:hi, h * G:(h + 1) * G] = torch.einsum("tgj,jd->tgd", w, v)
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(s, -1)
    return out, lse
