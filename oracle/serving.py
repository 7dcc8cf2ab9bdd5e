"""CPU oracle of the paged-serving operators -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; the CUDA library and its binding never
do, and this module imports nothing from them.  Plain definitions, one request,
token and head at a time, in fp64 (integers for the tables):

    page_plan        block tables, slot map and positions from lengths
    paged_attention  softmax attention over the positions each token sees
    sample           temperature, top-k, top-p, min-p, and the race of the kept
                     tokens against given exponential random numbers

The source's pages describe serving of one request ("Quantize the Target,
Quantize the Drafter", pith.science review); interface and layout are this
library's (include/w4a16.h).
"""
from __future__ import annotations

import numpy as np


def page_plan(past, new, free, table, page, tokens):
    """-> (table, q_start, kv_len, positions, slots, pages_used)."""
    table = np.array(table, dtype=np.int64)
    B, columns = table.shape
    positions, slots = np.full(tokens, -1), np.full(tokens, -1)
    q_start, kv_len, used, t = [0], [], 0, 0
    for b in range(B):
        p, n = max(int(past[b]), 0), max(int(new[b]), 0)
        held, need = -(-p // page), -(-(p + n) // page)
        for c in range(held, columns):
            at = used + c - held
            table[b, c] = free[at] if c < need and at < len(free) else -1
        for i in range(n):
            pos = p + i
            c = pos // page
            if c < columns:
                entry = table[b, c]
            else:
                entry = -1
            if t < tokens:
                positions[t] = pos
                slots[t] = entry * page + pos % page if entry >= 0 else -1
            t += 1
        used += need - held
        q_start.append(t)
        kv_len.append(p + n)
    return table, np.array(q_start), np.array(kv_len), positions, slots, used


def paged_attention(q, k_cache, v_cache, table, q_start, kv_len, window=0, block=False, scale=None):
    """q [T, Hq, d], caches [pages, Hkv, page, d] in fp64 -> (out, lse, spread),
    spread[t, h] = sum_j softmax_j |v_j| (for error bounds).  Rows of tokens
    past the last request stay NaN."""
    T, Hq, d = q.shape
    pages, Hkv, page, _ = k_cache.shape
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out = np.full((T, Hq, d), np.nan)
    spread = np.zeros((T, Hq, d))
    lse = np.full((T, Hq), np.nan)
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        L = min(int(kv_len[b]), table.shape[1] * page)
        for i in range(n):
            t = q_start[b] + i
            e = L - 1 if block else L - n + i
            lo = max(0, e - window + 1) if window else 0
            js = np.array([j for j in range(lo, e + 1) if 0 <= table[b, j // page] < pages], dtype=np.int64)
            out[t], lse[t] = 0.0, -np.inf
            if len(js) == 0:
                continue
            pg, sl = table[b, js // page], js % page
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                s = k_cache[pg, hk, sl] @ q[t, h] * scale
                m = s.max()
                w = np.exp(s - m)
                v = v_cache[pg, hk, sl]
                out[t, h] = w @ v / w.sum()
                spread[t, h] = w @ np.abs(v) / w.sum()
                lse[t, h] = m + np.log(w.sum())
    return out, lse, spread


def sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None):
    """One row: f32 logits [V], f32 noise [V] -> (token, logprob)."""
    x = np.asarray(logits, dtype=np.float32)
    greedy = temperature is not None and not temperature > 0
    t = np.float32(1.0 if temperature is None or greedy else temperature)
    with np.errstate(all="ignore"):
        z32 = x / t
    z = np.where(np.isnan(z32), -np.inf, z32.astype(np.float64))
    if z.max() == -np.inf:
        return -1, -np.inf
    p = np.exp(z - z.max())
    order = np.argsort(-z, kind="stable")
    order = order[z[order] > -np.inf]
    total = p.sum()
    if greedy:
        token = order[0]
    else:
        if top_k is not None and top_k > 0:
            order = order[:top_k]
        keep = np.ones(len(order), dtype=bool)
        if top_p is not None and top_p < 1:
            w = p[order]
            keep &= np.cumsum(w) - w < np.float32(top_p) * w.sum()
        if min_p is not None and min_p > 0:
            keep &= z[order] - z[order[0]] >= np.log(np.float64(np.float32(min_p)))
        keep[0] = True
        order = np.sort(order[keep])
        with np.errstate(divide="ignore"):
            score = z[order] - np.log(np.asarray(noise, dtype=np.float64)[order])
        token = order[np.argmax(score)]
    return int(token), float(z[token] - z.max() - np.log(total))
