"""GPU parity of rotary positions, the 8-bit cache and attention for drafted trees against the oracle (oracle/drafts.py,
oracle/serving.py, fp64).

Tolerances, from the arithmetic (half a step of bf16 is 2^-8 of a value, of fp16 2^-11, of f32 2^-24).

Rotation: sine and cosine are within 2^-22 of exact (an f32 of the angle's fraction of a turn, at most 2^-25 of a
turn off, and the function's own last places), the products and their sum add 3 * 2^-24 of |a| + |b|; one rounding
of the result.  With m the magnitude, for a pair (a, b):
    |y - ref| <= m 2^-21 (|a| + |b|) + u |ref|      (+ 2^-25 in fp16: half its smallest step)

Codes without a rotation are decided in IEEE binary32 on both sides: equal bits.  With one, the f32 key is within
e = m 2^-21 (|a| + |b|) of the oracle's, and a value next to a border may get the neighbouring code: the value that a
code stands for is within half a step and 2 e of the oracle's unrounded key.

Reading back: scale times code in f32 and one rounding: |x - ref| <= (u + 2^-23) |ref| (+ 2^-25).

Attention: softmax weights rounded once to the 16-bit type of the product with v (or kept in two parts: 2^-16), the
f32 scores, exponentials and sums within 2e-4 of exact for the sizes here (128 products in f32, scores below 64):
    |out - ref| <= (u_w + 2e-4) sum_j p_j |v_j| + u |ref|     (fp16: + n 2^-25 max|v| over a 16-bit cache, + 2^-25)
    |lse - ref| <= 1e-4 + 1e-6 |ref|
with u_w = 2^-8 for bf16, 2^-11 for fp16 over a 16-bit cache, 2^-15 for fp16 over an 8-bit one, whose weights go in two
parts (the long rows of the largest calls have one: test_drafts_edges.py).
"""
import numpy as np
import pytest
import torch

from oracle import drafts, serving
from test_serving import DT, Attn, f64, i32

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module")
def w():
    import int4_weight_only_gemm_gb300 as w
    return w


def partner_sum(x, n, inter):
    """|a| + |b| of the pair that each of the first 2 n columns is in, 0 for the others."""
    s, a = np.zeros_like(x), np.abs(x)
    if inter:
        both = a[..., 0:2 * n:2] + a[..., 1:2 * n:2]
        s[..., 0:2 * n:2] = s[..., 1:2 * n:2] = both
    else:
        both = a[..., :n] + a[..., n:2 * n]
        s[..., :n] = s[..., n:2 * n] = both
    return s


def positions_of(T, far, seed, skip=True):
    p = np.random.default_rng(seed).integers(0, far, T)
    p[0] = far - 1
    if skip and T > 4:
        p[2] = -1
        p[T - 1] = -2 ** 31
    return p


# ---------------------------------------------------------------------------
# rotary positions
# ---------------------------------------------------------------------------

# (tokens, heads, d, rotary, interleaved, far, dtype)
ROPE = [(1, 1, 64, 64, False, 100, "bf16"), (1, 40, 128, 128, False, 8448, "bf16"), (7, 5, 128, 128, True, 1 << 20, "fp16"),
        (64, 40, 128, 64, False, 131072, "bf16"), (33, 3, 256, 256, False, 131072, "fp16"), (33, 3, 256, 64, True, 4096, "bf16"),
        (700, 2, 64, 32, True, 2 ** 31 - 1, "bf16"), (129, 9, 128, 128, False, 2 ** 31 - 1, "fp16"),
        (50, 4, 128, 24, False, 5000, "bf16"), (50, 4, 128, 6, True, 5000, "fp16"), (20, 3, 72, 70, False, 5000, "bf16"),
        (20, 3, 8, 2, False, 5000, "bf16"), (20, 17, 200, 50, True, 5000, "fp16"), (3, 70, 128, 2, False, 999, "bf16")]


@pytest.mark.parametrize("case", range(len(ROPE)))
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_matches_oracle(w, case, inplace):
    T, H, d, rot, inter, far, dtype = ROPE[case]
    dt, r = DT[dtype], np.random.default_rng(case)
    f, m = drafts.frequencies(rot, scaling="ramp", factor=4.0, length=2048) if case % 2 else drafts.frequencies(rot)
    pos = positions_of(T, far, case)
    wide = torch.from_numpy(r.standard_normal((T, H + 3, d))).cuda().to(dt)   # a slice of wider rows
    kept, x = wide.clone(), wide[:, 2:2 + H]
    out = x if inplace else torch.full((T, H, d), 7.0, dtype=dt, device="cuda")
    res = w.w4a16_rope(x, i32(pos), torch.from_numpy(f).cuda(), interleaved=inter, magnitude=m, out=out)
    assert res is out
    x = f64(kept[:, 2:2 + H])
    ref = drafts.rotate(x, pos, f, inter, m)
    live = pos >= 0
    err = np.abs(f64(out) - ref)[live]
    bound = m * 2.0 ** -21 * partner_sum(x, rot // 2, inter) + U[dt] * np.abs(ref) + TINY[dt]
    # beyond 2^22 positions the f64 frequency's own last place counts, on both sides: 2^-53 of the angle each
    bound = bound + 2 * far * 2.0 ** -52 * partner_sum(x, rot // 2, inter) * m
    assert np.all(err <= bound[live])
    assert np.array_equal(f64(out)[live][..., rot:], x[live][..., rot:])
    assert torch.equal(out[torch.from_numpy(~live).cuda()], (kept[:, 2:2 + H] if inplace else torch.full_like(out, 7.0))[torch.from_numpy(~live).cuda()])
    assert torch.equal(wide[:, :2], kept[:, :2]) and torch.equal(wide[:, 2 + H:], kept[:, 2 + H:])


def test_rope_makes_an_output_and_takes_expanded_rows(w):
    x = torch.randn(1, 6, 128, device="cuda").to(torch.bfloat16).expand(9, 6, 128)
    f, _ = w.w4a16_rope_frequencies(128)
    pos = torch.arange(9, dtype=torch.int32, device="cuda")
    out = w.w4a16_rope(x, pos, f)
    ref = drafts.rotate(f64(x), range(9), f64(f))
    assert np.all(np.abs(f64(out) - ref) <= 2.0 ** -21 * partner_sum(f64(x), 64, False) + 2.0 ** -8 * np.abs(ref))
    assert torch.equal(out[0], x[0])
    empty = torch.empty(0, 6, 128, dtype=torch.bfloat16, device="cuda")
    assert w.w4a16_rope(empty, i32([]), f).shape == (0, 6, 128)


# ---------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------

def empty_cache(w, code, pages, H, page, d, order, dt):
    ct = CODE.get(code, dt)
    zero = lambda *s: torch.zeros(s, dtype=torch.int8 if code else torch.int16, device="cuda").view(ct)  # noqa: E731
    if order == "head":
        kc, vc = zero(2, pages, H, page, d)
        ks, vs = torch.zeros(2, pages, H, page, device="cuda")
    elif order == "slot":
        kc, vc = (c.transpose(1, 2) for c in zero(2, pages, page, H, d))
        ks, vs = (c.transpose(1, 2) for c in torch.zeros(2, pages, page, H, device="cuda"))
    else:
        both = zero(pages, 2, H, page, d)
        kc, vc = both[:, 0], both[:, 1]
        ks, vs = torch.zeros(pages, H, page, 2, device="cuda").unbind(-1)
    return kc, vc, (ks if code else None), (vs if code else None)


def by_slot(t):
    """[pages, H, page, ...] -> [slots, H, ...] on the host, 8-bit codes as bytes."""
    t = t.transpose(1, 2).contiguous()
    if t.dtype in (torch.int8, torch.float8_e4m3fn):
        t = t.view(torch.uint8)
    return t.reshape(-1, *t.shape[2:]).cpu().numpy() if t.dtype in (torch.uint8, torch.float32) else f64(t.reshape(-1, *t.shape[2:]))


# (tokens, kv heads, d, page, order, code, dtype)
STORE = [(1, 1, 64, 8, "head", "int8", "bf16"), (3, 8, 128, 16, "head", "e4m3", "bf16"), (64, 8, 128, 16, "slot", "int8", "fp16"),
         (517, 2, 64, 32, "both", "e4m3", "fp16"), (1000, 3, 16, 64, "head", "int8", "bf16"), (300, 5, 256, 16, "slot", "int8", "bf16"),
         (2049, 4, 128, 256, "slot", "e4m3", "bf16"), (33, 2, 144, 16, "both", "int8", "fp16")]


def some_slots(T, pages, page, r):
    slots = r.permutation(pages * page)[:T]
    slots[r.random(T) < 0.1] = -1
    if T > 10:
        slots[5], slots[6] = pages * page, 2 ** 31 - 1  # past the cache: skipped
    return slots, np.flatnonzero((slots >= 0) & (slots < pages * page))


@pytest.mark.parametrize("case", range(len(STORE)))
def test_write_quantises_by_the_definition(w, case):
    T, H, d, page, order, code, dtype = STORE[case]
    dt, r, pages = DT[dtype], np.random.default_rng(case), STORE[case][0] // page + 5
    x = r.standard_normal((2, T, H, d)) * np.exp(r.uniform(-4, 4, (2, T, H, 1)))
    if T > 20:
        x[0, 7, 0], x[1, 8, 0] = 0.0, 2.0 ** -24 * (dtype == "fp16")   # an empty row, a tiny one
        x[0, 9, 0, 3], x[1, 9, H - 1, d - 1], x[0, 10, 0, 0] = np.nan, np.inf, -np.inf
        x[0, 11, 0] = np.linspace(-63.5, 63.5, d)                      # many halves
    fused = torch.from_numpy(np.concatenate([x[0], x[1]], 1)).cuda().to(dt)
    k, v = fused[:, :H], fused[:, H:]
    kc, vc, ks, vs = empty_cache(w, code, pages, H, page, d, order, dt)
    slots, on = some_slots(T, pages, page, r)
    w.w4a16_kv_write(k, v, i32(slots), kc, vc, k_scale=ks, v_scale=vs)
    back = torch.full((2, T, H, d), 5.0, dtype=dt, device="cuda")
    w.w4a16_kv_read(kc, vc, i32(slots), back[0], back[1], k_scale=ks, v_scale=vs)
    for c, s, x, b in ((kc, ks, k, back[0]), (vc, vs, v, back[1])):
        codes, scale = drafts.quantise(x.float().cpu().numpy(), code)
        want, wants = np.zeros((pages * page, H, d), np.uint8), np.zeros((pages * page, H), np.float32)
        want[slots[on]], wants[slots[on]] = codes.view(np.uint8)[on], scale[on]
        assert np.array_equal(by_slot(c), want) and np.array_equal(by_slot(s), wants, equal_nan=True)
        ref, got = drafts.values(codes, scale, code)[on], f64(b)[on]
        assert np.array_equal(np.isnan(ref), np.isnan(got))
        fin = ~np.isnan(ref)
        assert np.all(np.abs(got - ref)[fin] <= (U[dt] + 2.0 ** -23) * np.abs(ref)[fin] + TINY[dt])
        assert (b[torch.from_numpy(np.setdiff1d(np.arange(T), on)).cuda()] == 5).all()


# (tokens, q heads, kv heads, d, rotary, interleaved, page, order, code, dtype)
TURNED = [(1, 4, 1, 64, 64, False, 16, "head", "int8", "bf16"), (64, 32, 8, 128, 128, False, 16, "head", "e4m3", "bf16"),
          (300, 6, 2, 128, 64, True, 64, "slot", "int8", "fp16"), (90, 0, 3, 128, 128, False, 32, "both", "int8", "bf16"),
          (77, 8, 2, 64, 24, False, 16, "both", None, "bf16"), (200, 12, 4, 128, 128, True, 128, "slot", None, "fp16"),
          (30, 5, 5, 256, 250, False, 8, "head", "e4m3", "bf16"), (513, 4, 4, 64, 64, True, 16, "head", "e4m3", "fp16")]


@pytest.mark.parametrize("case", range(len(TURNED)))
@pytest.mark.parametrize("inplace", [False, True])
def test_rope_kv_write_matches_oracle(w, case, inplace):
    T, Hq, H, d, rot, inter, page, order, code, dtype = TURNED[case]
    dt, r = DT[dtype], np.random.default_rng(100 + case)
    pages, pos = T // page + 5, positions_of(T, 40000, case)
    f, m = drafts.frequencies(rot, scaling="ramp", factor=2.0, length=4096)
    fused = torch.from_numpy(r.standard_normal((T, Hq + 2 * H, d))).cuda().to(dt)
    kept = fused.clone()
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:]
    kc, vc, ks, vs = empty_cache(w, code, pages, H, page, d, order, dt)
    slots, on = some_slots(T, pages, page, r)
    live = pos >= 0
    on = on[live[on]]
    out = None if not Hq else q if inplace else torch.full((T, Hq, d), 7.0, dtype=dt, device="cuda")
    res = w.w4a16_rope_kv_write(q if Hq else None, k, v, i32(pos), torch.from_numpy(f).cuda(), i32(slots), kc, vc, out, ks,
                                vs, inter, m)
    assert res is out and torch.equal(fused[:, Hq:], kept[:, Hq:])
    if Hq:
        x = f64(kept[:, :Hq])
        ref = drafts.rotate(x, pos, f, inter, m)
        bound = m * 2.0 ** -21 * partner_sum(x, rot // 2, inter) + U[dt] * np.abs(ref) + TINY[dt]
        assert np.all((np.abs(f64(out) - ref) <= bound)[live])
        dead = torch.from_numpy(~live).cuda()
        assert torch.equal(out[dead], (kept[:, :Hq] if inplace else torch.full_like(out, 7.0))[dead])
    x = f64(k)
    e = np.zeros((T, H, d)) + m * 2.0 ** -21 * partner_sum(x, rot // 2, inter)
    ref = drafts.rotate(x, pos, f, inter, m)
    off = np.setdiff1d(np.arange(pages * page), slots[on])
    if code is None:
        got = by_slot(kc)
        assert np.all(np.abs(got[slots[on]] - ref[on]) <= (e + U[dt] * np.abs(ref) + TINY[dt])[on])
        assert np.array_equal(by_slot(vc)[slots[on]], f64(v)[on]) and not got[off].any() and not by_slot(vc)[off].any()
        assert np.array_equal(got[slots[on]][..., rot:], x[on][..., rot:])
        return
    codes, scale = drafts.quantise(v.float().cpu().numpy(), code)
    assert np.array_equal(by_slot(vc)[slots[on]], codes.view(np.uint8)[on]) and np.array_equal(by_slot(vs)[slots[on]], scale[on])
    got = by_slot(kc)[slots[on]]
    got = got.view(np.int8) if code == "int8" else got
    kscale = by_slot(ks)[slots[on]]
    amax = np.abs(ref[on]).max(-1)
    assert np.all(np.abs(kscale * drafts.TOP[code] - amax) <= e[on].max(-1) + 2.0 ** -22 * amax)
    # half a step: of the grid, or 2^-4 of the value, down to half the smallest e4m3 step
    step = kscale[..., None].astype(np.float64) * (0.5 if code == "int8" else np.maximum(2.0 ** -4 * np.abs(ref[on] / kscale[..., None]), 2.0 ** -10))
    assert np.all(np.abs(drafts.values(got, kscale, code) - ref[on]) <= step * (1 + 1e-5) + 2 * e[on] + 2.0 ** -21 * amax[..., None])
    assert not by_slot(kc)[off].any() and not by_slot(ks)[off].any() and not by_slot(vc)[off].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_read_copies_a_16_bit_cache(w, dtype):
    dt, r = DT[dtype], np.random.default_rng(5)
    bits = torch.from_numpy(r.integers(-32768, 32768, (2, 9, 3, 16, 64)).astype(np.int16)).cuda()
    kc, vc = bits.view(dt)
    slots = np.concatenate([r.integers(0, 144, 200), [-1, 144]])   # the same slot more than once
    wide = torch.zeros(202, 10, 64, dtype=dt, device="cuda")
    k, v = wide[:, 1:4], wide[:, 5:8]
    assert w.w4a16_kv_read(kc, vc, i32(slots), k, v)[0] is k
    for x, c in ((k, bits[0]), (v, bits[1])):
        assert torch.equal(x[:200].contiguous().view(torch.int16), c.transpose(1, 2).reshape(144, 3, 64)[torch.from_numpy(slots[:200]).cuda()])
        assert (x[200:] == 0).all()
    assert (wide[:, 0] == 0).all() and (wide[:, 4] == 0).all() and (wide[:, 8:] == 0).all()


def test_every_code_reads_as_its_value(w):
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 16, 16)
    out = torch.empty(2, 16, 1, 16, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(1, 1, 16, device="cuda")
    ones[0, 0, 3] = float("inf")
    slots = torch.arange(16, dtype=torch.int32, device="cuda")
    for code, dt in CODE.items():
        c = codes.view(dt)
        w.w4a16_kv_read(c, c, slots, out[0], out[1], k_scale=ones, v_scale=ones)
        want = drafts.values(codes.cpu().numpy().reshape(16, 16).view(np.int8 if code == "int8" else np.uint8), ones.cpu().numpy()[0, 0], code)
        assert np.array_equal(f64(out[0, :, 0]), want, equal_nan=True) and torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Draft(Attn):
    """Requests over a cache of 16 or 8 bits, with a tree of each request's new tokens or without."""

    def __init__(self, lens, Hq, Hkv, d, page, dtype, code=None, tree=None, words=None, **kw):
        super().__init__(lens, Hq, Hkv, d, page, dtype, **kw)
        self.code, self.ks, self.vs, self.tree = code, None, None, None
        r = np.random.default_rng(kw.get("seed", 0) + 77)
        if code:
            caches = []
            for c in (self.kc, self.vc):
                x = c.float()
                codes, scale = drafts.quantise(np.where(np.isfinite(x.cpu().numpy()), x.cpu().numpy(), 0), code)
                scale = np.where(np.isfinite(x.cpu().numpy()).all(-1), scale * np.exp(r.uniform(-2, 2, scale.shape)), np.nan)
                caches.append((torch.from_numpy(codes.view(np.uint8)).cuda().view(CODE[code]),
                               torch.from_numpy(scale.astype(np.float32)).cuda()))
            (self.kc, self.ks), (self.vc, self.vs) = caches
            # scores of a few units: the scales of the keys vary by e^2 either way
            self.q = (self.q.float() * 0.3).to(self.dt)
        if tree:
            total = self.q.shape[0]
            rows = []
            for n in self.n:
                seen = []
                for i in range(n):
                    if tree == "tree":
                        up = i - 1 - int(r.random() ** 2 * 6)
                        seen.append((seen[up] if up >= 0 else []) + [i])
                    elif tree == "chain":
                        seen.append(list(range(i + 1)))
                    else:   # any bits: later nodes, none at all
                        seen.append([k for k in range(n) if r.random() < 0.3] if i % 5 else [])
                rows += seen
            rows += [[]] * (total - len(rows))
            self.words = -(-int(self.n.max()) // 32) if words is None else words
            self.tree = drafts.bits([[k for k in row if k < 32 * self.words] for row in rows], self.words)
            # bits past a request's nodes mean nothing
            junk = r.integers(0, 1 << 32, self.tree.shape, dtype=np.uint64).astype(np.uint32)
            at = np.arange(32 * self.words).reshape(self.words, 32)
            t = 0
            for n in self.n:
                keep = ((at < n).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
                for _ in range(n):
                    self.tree[t] = (self.tree[t].view(np.uint32) | (junk[t] & ~keep)).view(np.int32)
                    t += 1

    def run(self, w, window=0, **kw):
        more = dict(kw)
        if self.code:
            more.update(k_scale=self.ks, v_scale=self.vs)
        if self.tree is not None:
            more.setdefault("tree", i32(self.tree))
        return super().run(w, window, **more)

    def values(self):
        if not self.code:
            return f64(self.kc), f64(self.vc)
        return (drafts.values(c.contiguous().view(torch.uint8).cpu().numpy().view(np.int8 if self.code == "int8" else np.uint8),
                              s.cpu().numpy(), self.code) for c, s in ((self.kc, self.ks), (self.vc, self.vs)))

    def reference(self, window=0, block=False, scale=None):
        k, v = self.values()
        with np.errstate(all="ignore"):
            if self.tree is not None:
                return (*drafts.tree_attention(f64(self.q), k, v, self.table, self.q_start, self.L, self.tree, window, scale), v)
            return (*serving.paged_attention(f64(self.q), k, v, self.table, self.q_start, self.L, window, block, scale), v)

    def check(self, out, lse, window=0, block=False, scale=None, rows=None):
        ref, rl, spread, v = self.reference(window, block, scale)
        end = int(self.q_start[-1])
        ref, rl, spread, got, gl = ref[:end], rl[:end], spread[:end], f64(out)[:end], f64(lse)[:end]
        assert np.array_equal(np.isfinite(got), np.isfinite(ref)), "finite elsewhere than the definition"
        uw = 2.0 ** -8 if self.dt == torch.bfloat16 else 2.0 ** -15 if self.code else 2.0 ** -11
        bound = (uw + 2e-4) * spread + U[self.dt] * np.abs(ref) + TINY[self.dt]
        if self.dt == torch.float16 and not self.code:
            bound = bound + self.L.max() * 2.0 ** -25 * np.nanmax(np.where(np.isfinite(v), np.abs(v), 0))
        err = np.abs(got - ref)
        bad = ~(err <= bound) & np.isfinite(ref)
        assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, worst {np.nanmax(err / (bound + 1e-30)):.3g}, at {np.argwhere(bad)[:4].tolist()}"
        assert np.array_equal(np.isnan(gl), np.isnan(rl)) and np.array_equal(gl == -np.inf, rl == -np.inf)
        fin = np.isfinite(rl)
        assert np.all(np.abs(gl[fin] - rl[fin]) <= 1e-4 + 1e-6 * np.abs(rl[fin]))


# (requests (cached, new), Hq, Hkv, d, page, dtype, window, block)
CASES8 = [
    ([(0, 1)], 1, 1, 128, 16, "bf16", 0, False),
    ([(99, 1)], 32, 8, 128, 16, "bf16", 0, False),
    ([(2303, 1)], 8, 2, 128, 16, "fp16", 0, False),
    ([(1000, 1), (0, 1), (16, 1), (15, 1), (130, 1)], 8, 2, 64, 16, "fp16", 0, False),
    ([(500, 1), (40, 1), (1023, 1)], 14, 2, 128, 32, "bf16", 200, False),
    ([(700, 1), (64, 1)], 16, 1, 128, 64, "fp16", 0, False),
    ([(300, 1), (77, 1)], 34, 1, 64, 8, "bf16", 0, False),
    ([(300, 1), (5, 1)], 3, 1, 128, 8, "bf16", 0, False),
    ([(600, 4), (12, 4), (0, 4)], 16, 4, 128, 16, "bf16", 0, False),
    ([(1500, 16), (33, 16)], 16, 4, 128, 16, "bf16", 0, False),
    ([(1500, 16), (33, 16)], 8, 2, 128, 128, "bf16", 512, True),
    ([(0, 200)], 4, 2, 128, 16, "bf16", 0, False),
    ([(0, 257)], 3, 1, 64, 64, "fp16", 0, False),
    ([(333, 150)], 14, 2, 128, 256, "bf16", 0, False),
    ([(1000, 140), (0, 3), (250, 67)], 4, 1, 64, 8, "fp16", 100, False),
    ([(50, 129), (900, 1), (0, 0), (31, 1), (5, 12), (128, 128)], 8, 2, 128, 16, "bf16", 0, False),
    ([(50, 129), (900, 1), (0, 64), (31, 1)], 12, 4, 64, 32, "fp16", 70, False),
    ([(0, 130)], 64, 1, 64, 16, "bf16", 0, False),
    ([(5, 40), (300, 20)], 5, 5, 128, 16, "fp16", 0, True),
    ([(900, 90)], 2, 1, 128, 16, "bf16", 1, False),
]


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("case", range(len(CASES8)))
def test_attention_over_an_8_bit_cache(w, case, code):
    lens, Hq, Hkv, d, page, dtype, window, block = CASES8[case]
    a = Draft(lens, Hq, Hkv, d, page, dtype, code, seed=case)
    a.check(*a.run(w, window, block=block), window, block)
    assert w.w4a16_last_device_status() == 0


# (requests (cached, nodes), Hq, Hkv, d, page, dtype, window, masks)
TREES = [
    ([(0, 1)], 1, 1, 128, 16, "bf16", 0, "tree"),
    ([(99, 3)], 8, 2, 128, 16, "bf16", 0, "tree"),
    ([(2000, 4), (3, 2)], 16, 4, 128, 16, "bf16", 0, "tree"),
    ([(700, 16), (64, 9)], 4, 4, 64, 16, "fp16", 0, "any"),
    ([(300, 5), (9, 1)], 6, 2, 128, 8, "fp16", 40, "tree"),
    ([(1000, 13)], 32, 8, 128, 16, "bf16", 0, "tree"),
    ([(1500, 33), (0, 40), (127, 64)], 8, 2, 128, 32, "bf16", 0, "tree"),
    ([(500, 64), (63, 31), (0, 0), (5, 1)], 12, 4, 64, 64, "fp16", 100, "tree"),
    ([(300, 200)], 14, 2, 128, 16, "bf16", 0, "tree"),
    ([(100, 130), (40, 3)], 8, 2, 128, 256, "bf16", 64, "any"),
    ([(0, 150), (1, 100)], 4, 1, 64, 8, "fp16", 0, "any"),
    ([(250, 70)], 4, 1, 64, 16, "bf16", 0, "chain"),
    ([(33, 257)], 3, 1, 64, 64, "bf16", 16, "tree"),
    ([(60, 300)], 2, 2, 128, 16, "fp16", 0, "tree"),
]


@pytest.mark.parametrize("code", [None, "int8", "e4m3"])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_attention_of_a_tree(w, case, code):
    lens, Hq, Hkv, d, page, dtype, window, masks = TREES[case]
    a = Draft(lens, Hq, Hkv, d, page, dtype, code, masks, seed=case)
    a.check(*a.run(w, window), window)
    assert w.w4a16_last_device_status() == 0


def test_a_chain_is_causal_attention_and_masks_may_be_short_or_strided(w):
    for lens in ([(77, 3), (9, 4)], [(200, 70), (3, 40)]):
        a = Draft(lens, 8, 2, 128, 16, "bf16", tree="chain", seed=1, pad=3)
        out, lse = a.run(w)
        b = Draft(lens, 8, 2, 128, 16, "bf16", seed=1, pad=3)
        b.check(out, lse)
        # a wider mask's slice, and padding rows that stay
        wide = torch.full((a.tree.shape[0], a.words + 5), -1, dtype=torch.int32, device="cuda")
        wide[:, 2:2 + a.words] = i32(a.tree)
        res = torch.full_like(out, 3.0)
        again, lse2 = a.run(w, tree=wide[:, 2:2 + a.words], out=res)
        end = int(a.q_start[-1])
        assert torch.equal(again[:end], out[:end]) and torch.equal(lse2, lse) and (res[end:] == 3).all() and (lse2[end:] == 7).all()
    short = Draft([(200, 70)], 4, 2, 128, 16, "bf16", tree="tree", words=1, seed=2)   # nodes past the mask are not seen
    short.check(*short.run(w))


@pytest.mark.parametrize("order", ["slot", "both"])
@pytest.mark.parametrize("lens", [[(40, 1), (333, 1)], [(70, 150), (200, 9)]])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_8_bit_cache_strides(w, order, lens, code):
    a = Draft(lens, 8, 2, 128, 16, "bf16", code, seed=3, pad=5)
    pages = a.kc.shape[0]
    both = torch.stack([a.kc.view(torch.uint8), a.vc.view(torch.uint8)])
    both = both.transpose(2, 3).contiguous().transpose(2, 3) if order == "slot" else both.transpose(0, 1).contiguous().transpose(0, 1)
    a.kc, a.vc = both.view(CODE[code]) if order == "slot" else both.view(CODE[code]).unbind(0)
    a.ks, a.vs = a.ks.transpose(0, 2).contiguous().transpose(0, 2), torch.stack([a.vs, a.vs], -1)[..., 0]
    T = a.q.shape[0]
    wide = torch.zeros(T, 20, 128, dtype=a.dt, device="cuda")
    wide[:, 6:14] = a.q
    a.q = wide[:, 6:14]
    res = torch.full((T, 11, 128), 3.0, dtype=a.dt, device="cuda")
    out, lse = a.run(w, scale=0.05, max_q=1000, out=res[:, 2:10])
    a.check(out, lse, scale=0.05)
    end = int(a.q_start[-1])
    assert (res[:, :2] == 3).all() and (res[:, 10:] == 3).all() and (res[end:] == 3).all() and (lse[end:] == 7).all()
    # one scale for all
    a.ks, a.vs = torch.full((1, 1, 1), 0.02, device="cuda").expand(pages, 2, 16), torch.full((1, 2, 1), 0.5, device="cuda").expand(pages, 2, 16)
    a.check(*a.run(w))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("fill", ["bits", "nan", "inf"])
@pytest.mark.parametrize("lens,window,tree", [([(99, 1), (17, 1)], 0, None), ([(99, 1), (300, 1)], 40, None),
                                              ([(40, 150), (3, 60)], 0, None), ([(333, 16)], 0, None), ([(500, 130)], 64, None),
                                              ([(30, 4), (77, 2)], 0, "tree"), ([(90, 70)], 20, "tree")])
def test_8_bit_attention_ignores_what_pages_held_before(w, fill, lens, window, tree, code):
    """Slots behind a request's positions hold any codes and scales."""
    a = Draft(lens, 8, 2, 128, 16, "bf16", code, tree, seed=5)
    used = torch.zeros(a.ks.shape[0], 16, dtype=torch.bool)
    for b, L in enumerate(a.L):
        for j in range(int(L)):
            used[a.table[b, j // 16], j % 16] = True
    free = ~used[:, None].expand(-1, 2, -1).cuda()
    for c, s in ((a.kc, a.ks), (a.vc, a.vs)):
        c.view(torch.uint8)[free] = 0x7f if fill != "bits" else 0xff
        s[free] = {"bits": 3e38, "nan": float("nan"), "inf": float("-inf")}[fill]
    a.check(*a.run(w, window), window)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("lens,pos,window,tree", [([(30, 150)], 100, 0, None), ([(0, 20)], 7, 0, None), ([(300, 140)], 290, 64, None),
                                                  ([(64, 5)], 66, 0, None), ([(200, 300)], 255, 0, None), ([(900, 1)], 300, 400, None),
                                                  ([(900, 1)], 600, 400, None), ([(100, 4)], 102, 0, "tree"), ([(100, 60)], 120, 0, "tree"),
                                                  ([(300, 60)], 20, 0, "tree")])
def test_a_bad_scale_reaches_the_tokens_that_see_it(w, bad, where, code, lens, pos, window, tree):
    a = Draft(lens, 8, 2, 128, 16, "bf16", code, tree, seed=6)
    (a.ks if where == "k" else a.vs)[int(a.table[0, pos // 16]), 1, pos % 16] = bad
    out, lse = a.run(w, window)
    assert torch.isnan(out).any() == bool(np.isnan(a.reference(window)[0]).any())
    if where == "k":
        a.check(out, lse, window)
        return
    # a value of NaN leaves the log-sum alone
    ref, rl, spread, _ = a.reference(window)
    seen = np.isnan(ref)
    got = f64(out)
    assert np.array_equal(np.isnan(got), seen)
    assert np.all((np.abs(got - ref) <= (2.0 ** -8 + 2e-4) * spread + 2.0 ** -8 * np.abs(ref))[~seen])
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4 + 1e-6 * np.abs(rl))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("lens,pos", [([(100, 4)], 102), ([(100, 60)], 120), ([(300, 60)], 301), ([(10, 200)], 205), ([(5, 3)], 2)])
def test_a_bad_node_reaches_the_paths_through_it(w, bad, where, lens, pos):
    """16-bit cache: a NaN or an infinity at one node reaches its descendants, and no other path."""
    a = Draft(lens, 8, 2, 128, 16, "bf16", tree="tree", seed=7)
    clean = Draft(lens, 8, 2, 128, 16, "bf16", tree="tree", seed=7)
    (a.kc if where == "k" else a.vc)[int(a.table[0, pos // 16]), 1, pos % 16, 3] = bad
    out, lse = a.run(w)
    ref, rl, spread, _ = clean.reference()
    k = pos - lens[0][0]
    sees = np.array([k < 0 or bool(int(row.view(np.uint32)[k // 32]) >> (k % 32) & 1) for row in a.tree])
    hit = sees[:, None] & (np.arange(8) >= 4)[None]
    got, bound = f64(out), (2.0 ** -8 + 2e-4) * spread + 2.0 ** -8 * np.abs(ref)
    assert np.all((np.abs(got - ref) <= bound)[~hit]) and np.all(np.abs(f64(lse) - rl)[~hit] <= 1e-4)
    if where == "v":
        assert not np.isfinite(got[hit][:, 3]).any()
        cols = np.arange(128) != 3
        assert np.all((np.abs(got - ref) <= bound)[hit][:, cols])
    elif np.isnan(bad):
        assert np.isnan(got[hit]).all()


@pytest.mark.parametrize("code,tree", [("int8", None), ("e4m3", "any"), (None, "any"), ("int8", "tree")])
def test_rows_without_a_position(w, code, tree):
    a = Draft([(0, 20), (100, 1), (60, 40), (30, 1), (0, 1)], 8, 2, 128, 16, "bf16", code, tree, seed=8)
    a.L[0] = 6            # nodes or tokens before the cache's first position
    a.table[1, :] = -1    # no page at all
    a.table[2, 2] = 1 << 20
    a.table[2, 4] = -7
    a.L[4] = 0
    out, lse = a.run(w)
    a.check(out, lse)
    assert (out[20] == 0).all() and (lse[20] == -np.inf).all() and (out[-1] == 0).all()
    a.L[3] = 10 ** 9      # longer than its table: counted as the table's room
    out, lse = a.run(w, window=50)
    a.check(out, lse, window=50)


def test_scales_far_apart(w):
    """Values a billion times larger than others, seen with small weight and large."""
    for lens in ([(200, 1)], [(200, 30)]):
        for dtype in ("bf16", "fp16"):
            a = Draft(lens, 8, 2, 128, 16, dtype, "int8", seed=9)
            a.vs *= 1e-3
            big = torch.rand(a.vs.shape, device="cuda") < 0.02
            a.vs[big] *= 2.0 ** (30 if dtype == "bf16" else 12)
            a.check(*a.run(w))


def test_deterministic_streams_and_workspace(w):
    for lens, tree in (([(3000, 1), (50, 1)], None), ([(900, 130), (10, 1), (77, 16)], None), ([(2000, 4)], "tree"), ([(900, 70), (10, 3)], "tree")):
        for code in (None, "int8"):
            if not (code or tree):
                continue
            a = Draft(lens, 8, 2, 128, 16, "bf16", code, tree, seed=10)
            need = w.w4a16_paged_attention_workspace_bytes(a.q.shape[0], len(lens), 8, 2, 128, int(a.n.max()))
            ws = w.new_workspace(max(need, 1 << 17))
            first, l1 = a.run(w, workspace=ws)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            again, l2 = a.run(w, workspace=ws, stream=s, flags=0)
            s.synchronize()
            assert torch.equal(first, again) and torch.equal(l1, l2)
            assert ws[:65536].view(torch.int32).abs().sum().item() == 0


def test_argument_errors(w):
    a = Draft([(20, 3)], 8, 2, 128, 16, "bf16", "int8", seed=0)
    call = lambda **kw: w.w4a16_paged_attention(**{**dict(  # noqa: E731
        q=a.q, k_cache=a.kc, v_cache=a.vc, block_table=i32(a.table), q_start=i32(a.q_start), kv_len=i32(a.L), max_q=3,
        k_scale=a.ks, v_scale=a.vs), **kw})
    call()
    tree = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    for kw in (dict(k_scale=None), dict(v_scale=None), dict(k_scale=None, v_scale=None), dict(k_scale=a.ks.double()),
               dict(k_scale=a.ks[:, :1]), dict(v_scale=a.vs.cpu()), dict(v_cache=a.vc.view(torch.float8_e4m3fn)),
               dict(k_cache=a.kc.view(torch.uint8), v_cache=a.vc.view(torch.uint8)), dict(tree=tree[:2]), dict(tree=tree.long()),
               dict(tree=tree[:, :0]), dict(tree=tree.cpu()), dict(q=a.q.float())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(w.W4A16Error):
        call(tree=tree, block=True)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = i32([0, 1, 2])
    for kw in (dict(k_scale=a.ks), dict(k_scale=a.ks, v_scale=a.vs[:1]), dict()):
        with pytest.raises(ValueError):
            w.w4a16_kv_write(k, k, slots, a.kc, a.vc, **kw)
    f, _ = w.w4a16_rope_frequencies(128)
    for bad in (f.float(), f.cpu(), f[::2], f[None]):
        with pytest.raises(ValueError):
            w.w4a16_rope(k, slots, bad)
    with pytest.raises(w.W4A16Error):
        w.w4a16_rope(k, slots, w.w4a16_rope_frequencies(256)[0])
