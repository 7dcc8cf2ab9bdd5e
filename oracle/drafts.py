"""CPU oracle of rotary positions, the 8-bit cache and attention for drafted trees -- TEST INFRASTRUCTURE ONLY.

Only ``tests/`` may import this module; the CUDA library and its binding never
do, and this module imports nothing from them.  Plain definitions in fp64:

    rotate           rotary positions of [T, heads, d]
    frequencies      radians per position, by scaling
    quantise         codes and scales of rows, decided in IEEE binary32
    values           what codes and scales stand for
    tree_attention   softmax attention of a tree's nodes over the context and their paths

The source's pages describe drafting and verification of one request ("Quantize
the Target, Quantize the Drafter", pith.science review); interface and layout
are this library's (include/w4a16.h).
"""
from __future__ import annotations

import math

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}


def rotate(x, positions, freq, interleaved=False, magnitude=1.0):
    """x [T, heads, d] in fp64; rows of negative positions stay."""
    y = np.array(x, dtype=np.float64)
    n = len(freq)
    for t, p in enumerate(positions):
        if p < 0:
            continue
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
            # the angle in turns: the whole ones of a position go away in integers
            turns = float(freq[i]) / (2 * math.pi)
            w = 2 * math.pi * math.fmod(math.fmod(turns, 1.0) * float(p), 1.0)
            c, s = math.cos(w) * magnitude, math.sin(w) * magnitude
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, a] * s + x[t, :, b] * c
    return y


def frequencies(r, base=10000.0, scaling="none", factor=1.0, length=0.0, low=1.0, high=32.0):
    """-> (radians per position [r / 2], magnitude)."""
    plain = [base ** (-2.0 * i / r) for i in range(r // 2)]
    if scaling == "none":
        return np.array(plain), 1.0
    if scaling == "linear":
        return np.array(plain) / factor, 1.0
    if scaling == "base":
        wide = base * factor ** (r / (r - 2.0)) if r > 2 else base
        return np.array([wide ** (-2.0 * i / r) for i in range(r // 2)]), 1.0
    if scaling == "ramp":
        pair = lambda turns: r * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        # the line's ends are whole pairs, the last of which may lie behind the head's (there are r // 2)
        first, last = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), r - 1)
        share = [1.0 if i >= last else max((i - first) / max(last - first, 1), 0.0) for i in range(r // 2)]
        return np.array([f * (1 - s) + f / factor * s for f, s in zip(plain, share)]), 0.1 * math.log(factor) + 1.0
    out = []
    for f in plain:
        turns = length * f / (2 * math.pi)
        kept = min(max((turns - low) / (high - low), 0.0), 1.0)
        out.append(f * kept + f / factor * (1 - kept))
    return np.array(out), 1.0


def e4m3_value(code):
    """The value of e4m3 codes 0 .. 255; the two without one count as +-480, as any other bits would say."""
    code = np.asarray(code, dtype=np.int64)
    e, m, sign = (code >> 3) & 15, code & 7, np.where(code & 128, -1.0, 1.0)
    return sign * np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))


_E4M3 = e4m3_value(np.arange(127))  # 0 .. 448, rising


def _e4m3_code(y):
    """Nearest e4m3 code of f32 values up to 448 and a rounding error, ties to the even code."""
    a = np.minimum(np.abs(y.astype(np.float64)), 448.0)
    hi = np.clip(np.searchsorted(_E4M3, a), 1, 126)
    lo = hi - 1
    up, down = _E4M3[hi] - a, a - _E4M3[lo]
    code = np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code + np.where(np.signbit(y), 128, 0)).astype(np.uint8)


def quantise(x, code):
    """Rows x [..., d] in f32 -> (codes: int8 or uint8, scales f32 [...])."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)
        bad, none = ~np.isfinite(x).all(-1), amax < np.float32(2.0 ** -100)
        top = np.float32(TOP[code])
        scale = np.where(bad, np.float32(np.nan), np.where(none, np.float32(0), amax / top))
        inv = np.where(bad | none, np.float32(0), top / amax).astype(np.float32)
        y = np.where(bad[..., None], np.float32(0), x) * inv[..., None]
    return (np.rint(y).astype(np.int8) if code == "int8" else _e4m3_code(y)), scale.astype(np.float32)


def values(codes, scales, code):
    """What codes stand for, in fp64; a scale that is not finite stands for NaN."""
    c = codes.astype(np.float64) if code == "int8" else e4m3_value(codes.view(np.uint8))
    s = np.where(np.isfinite(scales), scales.astype(np.float64), np.nan)
    return c * s[..., None]


def bits(paths, words):
    """Lists of the nodes that each row sees -> int32 [rows, words]."""
    m = np.zeros((len(paths), words), dtype=np.uint32)
    for t, path in enumerate(paths):
        for k in path:
            m[t, k // 32] |= np.uint32(1 << (k % 32))
    return m.view(np.int32)


def tree_attention(q, k_cache, v_cache, table, q_start, kv_len, tree, window=0, scale=None):
    """q [T, Hq, d], caches [pages, Hkv, page, d] in fp64, tree int32 [T, words] -> (out, lse, spread) as
    serving.paged_attention gives them."""
    T, Hq, d = q.shape
    pages, Hkv, page, _ = k_cache.shape
    scale = 1.0 / np.sqrt(d) if scale is None else scale
    out, spread, lse = np.full((T, Hq, d), np.nan), np.zeros((T, Hq, d)), np.full((T, Hq), np.nan)
    mask = tree.view(np.uint32)
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        L = min(int(kv_len[b]), table.shape[1] * page)
        past = L - n
        for t in range(q_start[b], q_start[b + 1]):
            nodes = [k for k in range(min(n, 32 * mask.shape[1])) if int(mask[t, k // 32]) >> (k % 32) & 1]
            first = max(0, past + len(nodes) - window) if window else 0
            js = list(range(first, past)) + [past + k for k in nodes if past + k >= 0]
            js = np.array([j for j in js if 0 <= table[b, j // page] < pages], dtype=np.int64)
            out[t], lse[t] = 0.0, -np.inf
            if len(js) == 0:
                continue
            pg, sl = table[b, js // page], js % page
            for h in range(Hq):
                hk = h // (Hq // Hkv)
                s = k_cache[pg, hk, sl] @ q[t, h] * scale
                m = s.max()
                p = np.exp(s - m)
                v = v_cache[pg, hk, sl]
                out[t, h] = p @ v / p.sum()
                spread[t, h] = p @ np.abs(v) / p.sum()
                lse[t, h] = m + np.log(p.sum())
    return out, lse, spread
