"""GPU parity of the paged-serving operators against the oracle
(oracle/serving.py, fp64; integers for the tables).

Tolerances, from the arithmetic.  Attention: the softmax weights are rounded
once to the inputs' type (relative u: 2^-9 for bf16, 2^-12 for fp16, plus half
the smallest fp16 subnormal, 2^-25, a weight), the result once (u |out|), and
the f32 scores, exponentials and sums are within 2e-4 of exact for the sizes
here (128 products of a score in f32, scores below 64 in magnitude):

    |out - ref| <= (u + 2e-4) sum_j p_j |v_j| + u |ref| + n 2^-25 max|v| (fp16)
    |lse - ref| <= 1e-4 + 1e-6 |ref|

Integers and copies are exact.  Sampling: tokens exact; |logprob - ref| <= 2e-5
+ 2e-6 |ref| (an f32 division, exponentials and a sum of non-negative terms).
"""
import numpy as np
import pytest
import torch

from oracle import serving

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def w():
    import int4_weight_only_gemm_gb300 as w
    return w


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def f64(t):
    return t.double().cpu().numpy()


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------

def plan_case(B, page, seed, past_max, new_max, spare=5, cut=0, pad=7):
    r = np.random.default_rng(seed)
    past = r.integers(0, past_max + 1, B)
    new = r.integers(0, new_max + 1, B)
    if B > 3:
        past[1], new[2] = 0, 0          # a fresh request, and one that rests
        past[3] = page * max(1, past_max // page)  # a full last page
    columns = int((-(-(past + new) // page)).max()) + 2 - cut
    table = r.integers(0, 1 << 20, (B, columns))
    free = r.permutation(1 << 12)[:max(0, int((-(-(past + new) // page) + -past // page).sum()) + spare)]
    return past, new, free, table, int(new.sum()) + pad


@pytest.mark.parametrize("B,page,past_max,new_max,spare,cut", [
    (1, 16, 0, 1, 5, 0), (1, 8, 300, 1, 0, 0), (2, 256, 1000, 700, 5, 0), (5, 16, 50, 40, 5, 0),
    (64, 16, 2000, 1, 5, 0), (97, 32, 500, 33, -40, 0),   # too few free pages
    (33, 16, 400, 20, 5, 4),                              # a table too narrow for the longest
    (513, 64, 900, 9, 5, 0), (2500, 16, 60, 3, 5, 0), (16384, 128, 200, 2, 5, 0)])
def test_plan_matches_oracle(w, B, page, past_max, new_max, spare, cut):
    past, new, free, table, T = plan_case(B, page, B + page, past_max, new_max, spare, cut)
    t = i32(table)
    q_start, kv_len, pos, slots, used = w.w4a16_page_plan(i32(past), i32(new), i32(free), t, page, max_tokens=T)
    ref = serving.page_plan(past, new, free, table, page, T)
    for got, want, what in zip((t, q_start, kv_len, pos, slots, used), ref, ("table", "q_start", "kv_len", "positions",
                                                                            "slots", "used")):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(want).ravel()), what
    # again on its own output: the entries it filled are filled the same way
    w.w4a16_page_plan(i32(past), i32(new), i32(free), t, page, q_start, kv_len, pos, slots, used)
    assert np.array_equal(t.cpu().numpy(), ref[0])


def test_plan_strided_table_negative_lengths_and_fewer_tokens(w):
    past, new = np.array([5, -3, 20]), np.array([3, 9, -1])
    wide = torch.full((3, 12), 77, dtype=torch.int32, device="cuda")
    free = np.arange(100, 110)
    out = w.w4a16_page_plan(i32(past), i32(new), i32(free), wide[:, 2:8], 8, max_tokens=6)
    ref = serving.page_plan(past, new, free, np.full((3, 6), 77), 8, 6)
    assert np.array_equal(wide[:, 2:8].cpu().numpy(), ref[0])
    assert (wide[:, :2] == 77).all() and (wide[:, 8:] == 77).all()
    for got, want in zip(out, ref[1:]):
        assert np.array_equal(got.cpu().numpy().ravel(), np.asarray(want).ravel())


def test_plan_empty_batch(w):
    empty = i32(np.zeros(0))
    q_start, _, pos, slots, used = w.w4a16_page_plan(empty, empty, empty, i32(np.zeros((0, 4))), 16, max_tokens=3)
    assert q_start.tolist() == [0] and used.tolist() == [0] and slots.tolist() == [-1] * 3 == pos.tolist()


# ---------------------------------------------------------------------------
# cache write
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T,H,d,page,order", [
    (1, 1, 64, 8, "head"), (3, 8, 128, 16, "head"), (64, 8, 128, 16, "slot"), (517, 2, 64, 32, "both"),
    (1000, 3, 8, 64, "head"), (2049, 4, 128, 256, "slot")])
def test_write_copies_bits(w, T, H, d, page, order, dtype):
    dt = DT[dtype]
    r = np.random.default_rng(T + H)
    pages = T // page + 5
    bits = torch.from_numpy(r.integers(-32768, 32768, (T, 3 * H * d + 8)).astype(np.int16)).cuda()  # NaN bits too
    fused = bits.view(dt)
    k, v = fused[:, 8:8 + H * d].view(T, H, d), fused[:, 8 + 2 * H * d:].view(T, H, d)
    if order == "head":      # [page][head][slot][d]
        kc, vc = torch.zeros(2, pages, H, page, d, dtype=dt, device="cuda")
    elif order == "slot":    # [page][slot][head][d]
        kc, vc = (c.transpose(1, 2) for c in torch.zeros(2, pages, page, H, d, dtype=dt, device="cuda"))
    else:                    # keys and values of a page side by side
        both = torch.zeros(pages, 2, H, page, d, dtype=dt, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    slots = r.permutation(pages * page)[:T]
    slots[r.random(T) < 0.1] = -1
    if T > 10:
        slots[5] = pages * page  # past the cache: skipped
    want = [np.zeros((pages * page, H, d), np.int16) for _ in range(2)]
    for x, c in zip(want, (k, v)):
        on = (slots >= 0) & (slots < pages * page)
        x[slots[on]] = c.contiguous().view(torch.int16).cpu().numpy()[on]
    w.w4a16_kv_write(k, v, i32(slots), kc, vc)
    for x, c in zip(want, (kc, vc)):
        got = c.transpose(1, 2).contiguous().view(torch.int16).cpu().numpy().reshape(pages * page, H, d)
        assert np.array_equal(got, x)


def test_write_on_another_stream(w):
    k, v = torch.randn(2, 40, 4, 64, device="cuda").to(torch.bfloat16)
    kc, vc = torch.zeros(2, 6, 4, 16, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    slots = torch.arange(40, dtype=torch.int32, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    w.w4a16_kv_write(k, v, slots, kc, vc, stream=s)
    s.synchronize()
    assert torch.equal(kc.transpose(1, 2).reshape(96, 4, 64)[:40], k)
    assert torch.equal(vc.transpose(1, 2).reshape(96, 4, 64)[:40], v)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Attn:
    def __init__(self, lens, Hq, Hkv, d, page, dtype, seed=0, order="head", pad=0, fill=None, qscale=1.0):
        """lens: (cached before, new) of each request; the caches start out full of `fill` (random if None)."""
        r = np.random.default_rng(seed)
        self.dt, self.page, self.Hq, self.Hkv, self.d = DT[dtype], page, Hq, Hkv, d
        past, new = np.array(lens, dtype=np.int64).T
        self.n, self.L = new, past + new
        held = -(-self.L // page)
        pages = int(held.sum()) + 3
        columns = int(held.max()) + 1
        order_of = r.permutation(pages)
        self.table = np.full((len(lens), columns), -1)
        at = 0
        for b, h in enumerate(held):
            self.table[b, :h] = order_of[at:at + h]
            at += h
        self.q_start = np.concatenate([[0], np.cumsum(new)])
        T = int(self.q_start[-1]) + pad
        q = torch.from_numpy(r.standard_normal((T, Hq, d)) * qscale).cuda().to(self.dt)
        self.q = q
        kv = torch.from_numpy(r.standard_normal((2, pages, Hkv, page, d))).cuda().to(self.dt)
        if fill is not None:  # only the requests' own positions hold numbers
            full = torch.full_like(kv, fill)
            for b in range(len(lens)):
                for c in range(held[b]):
                    n = min(page, int(self.L[b]) - c * page)
                    full[:, self.table[b, c], :, :n] = kv[:, self.table[b, c], :, :n]
            kv = full
        if order == "slot":
            kv = kv.transpose(2, 3).contiguous().transpose(2, 3)
        elif order == "both":
            kv = kv.transpose(0, 1).contiguous().transpose(0, 1)
        self.kc, self.vc = kv[0], kv[1]

    def run(self, w, window=0, block=False, scale=None, max_q=None, **kw):
        lse = torch.full((self.q.shape[0], self.Hq), 7.0, device="cuda")
        out = w.w4a16_paged_attention(self.q, self.kc, self.vc, i32(self.table), i32(self.q_start), i32(self.L),
                                      int(self.n.max()) if max_q is None else max_q, window, block, scale, lse=lse, **kw)
        return out, lse

    def check(self, out, lse, window=0, block=False, scale=None, kc=None, vc=None):
        kc, vc = f64(self.kc if kc is None else kc), f64(self.vc if vc is None else vc)
        ref, rl, spread = serving.paged_attention(f64(self.q), kc, vc, self.table, self.q_start, self.L, window,
                                                  block, scale)
        end = int(self.q_start[-1])
        ref, rl, spread = ref[:end], rl[:end], spread[:end]
        got, gl = f64(out)[:end], f64(lse)[:end]
        assert np.array_equal(np.isfinite(got), np.isfinite(ref)), "finite elsewhere than the definition"
        u = 2.0 ** -9 if self.dt == torch.bfloat16 else 2.0 ** -12
        bound = (u + 2e-4) * spread + u * np.abs(ref)
        if self.dt == torch.float16:
            bound = bound + self.L.max() * 2.0 ** -25 * np.nanmax(np.where(np.isfinite(vc), np.abs(vc), 0))
        err = np.abs(got - ref)
        bad = ~(err <= bound) & np.isfinite(ref)
        assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, worst {np.nanmax(err / (bound + 1e-30)):.3g}, at {np.argwhere(bad)[:4].tolist()}"
        assert np.array_equal(gl == -np.inf, rl == -np.inf)
        fin = np.isfinite(rl)
        assert np.all(np.abs(gl[fin] - rl[fin]) <= 1e-4 + 1e-6 * np.abs(rl[fin]))


# (requests (cached, new), Hq, Hkv, d, page, dtype, window, block)
ATTN = [
    ([(0, 1)], 1, 1, 128, 16, "bf16", 0, False),                       # the first token of all
    ([(99, 1)], 32, 8, 128, 16, "bf16", 0, False),
    ([(2303, 1)], 8, 2, 128, 16, "bf16", 0, False),                    # one long request: split over the GPU
    ([(1000, 1), (0, 1), (16, 1), (15, 1), (130, 1)], 8, 2, 64, 16, "fp16", 0, False),
    ([(500, 1), (40, 1), (1023, 1)], 14, 2, 128, 32, "bf16", 200, False),
    ([(700, 1), (64, 1)], 16, 1, 128, 64, "fp16", 0, False),           # sixteen heads on one key head
    ([(300, 1), (77, 1)], 34, 1, 64, 8, "bf16", 0, False),             # more rows than a small tile holds
    ([(600, 4), (12, 4), (0, 4)], 16, 4, 128, 16, "bf16", 0, False),   # short draft blocks
    ([(1500, 16), (33, 16)], 16, 4, 128, 16, "bf16", 0, False),        # 16-token blocks
    ([(1500, 16), (33, 16)], 8, 2, 128, 128, "bf16", 512, True),       # all tokens of a block see it
    ([(0, 200)], 4, 2, 128, 16, "bf16", 0, False),                     # a whole prompt
    ([(0, 257)], 3, 1, 64, 64, "fp16", 0, False),                      # an odd group
    ([(333, 150)], 14, 2, 128, 256, "bf16", 0, False),                 # a chunk, seven heads a group
    ([(1000, 140), (0, 3), (250, 67)], 4, 1, 64, 8, "fp16", 100, False),
    ([(50, 129), (900, 1), (0, 0), (31, 1), (5, 12), (128, 128)], 8, 2, 128, 16, "bf16", 0, False),  # a mixed step
    ([(50, 129), (900, 1), (0, 64), (31, 1)], 12, 4, 64, 32, "fp16", 70, False),
    ([(0, 130)], 64, 1, 64, 16, "bf16", 0, False),                     # 64 heads on one key head
    ([(5, 40), (300, 20)], 5, 5, 128, 16, "bf16", 0, True),            # a head group of one
    ([(3000, 90)], 2, 1, 128, 16, "bf16", 1, False),                   # each token sees itself
]


@pytest.mark.parametrize("case", range(len(ATTN)))
def test_attention_matches_oracle(w, case):
    lens, Hq, Hkv, d, page, dtype, window, block = ATTN[case]
    a = Attn(lens, Hq, Hkv, d, page, dtype, seed=case)
    a.check(*a.run(w, window, block), window, block)
    assert w.w4a16_last_device_status() == 0


@pytest.mark.parametrize("order", ["slot", "both"])
@pytest.mark.parametrize("lens", [[(40, 1), (333, 1)], [(70, 150), (200, 9)]])
def test_attention_strides(w, order, lens):
    """Token-major pages, keys beside values, q and out as slices of wider rows, a scale, a loose max_q, padding rows."""
    a = Attn(lens, 8, 2, 128, 16, "bf16", seed=3, order=order, pad=5)
    T = a.q.shape[0]
    wide = torch.zeros(T, 20, 128, dtype=a.dt, device="cuda")
    wide[:, 6:14] = a.q
    a.q = wide[:, 6:14]
    res = torch.full((T, 11, 128), 3.0, dtype=a.dt, device="cuda")
    out, lse = a.run(w, scale=0.05, max_q=1000, out=res[:, 2:10])
    a.check(out, lse, scale=0.05)
    end = int(a.q_start[-1])
    assert (res[:, :2] == 3).all() and (res[:, 10:] == 3).all() and (res[end:] == 3).all() and (lse[end:] == 7).all()


@pytest.mark.parametrize("fill", [float("nan"), float("inf"), -65504.0])
@pytest.mark.parametrize("lens,window", [([(99, 1), (17, 1)], 0), ([(99, 1), (300, 1)], 40),
                                         ([(40, 150), (3, 60)], 0), ([(333, 16)], 0), ([(500, 130)], 64)])
def test_attention_ignores_what_pages_held_before(w, fill, lens, window):
    a = Attn(lens, 8, 2, 128, 16, "bf16", seed=5, fill=fill)
    a.check(*a.run(w, window), window)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("lens,pos,window", [([(30, 150)], 100, 0), ([(0, 20)], 7, 0), ([(300, 140)], 290, 64),
                                             ([(64, 5)], 66, 0), ([(200, 300)], 255, 0), ([(900, 1)], 300, 400)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_attention_tokens_that_do_not_see_a_bad_position(w, bad, lens, pos, window, where):
    """A NaN or an infinity at one position reaches the tokens that see it, and no others."""
    a = Attn(lens, 8, 2, 128, 16, "bf16", seed=6)
    c = a.kc if where == "k" else a.vc
    c[int(a.table[0, pos // 16]), 1, pos % 16, 3] = bad
    out, lse = a.run(w, window)
    e = a.L[0] - a.n[0] + np.arange(a.n[0])
    hidden = (e < pos) | ((e - window + 1 > pos) if window else False)
    clean = Attn(lens, 8, 2, 128, 16, "bf16", seed=6)
    got, gl = f64(out), f64(lse)
    ref, rl, spread = serving.paged_attention(f64(clean.q), f64(clean.kc), f64(clean.vc), a.table, a.q_start, a.L, window)
    ok = hidden[:, None] | (np.arange(8) < 4)[None]  # tokens that do not see it, and the other key head
    bound = (2.0 ** -9 + 2e-4) * spread + 2.0 ** -9 * np.abs(ref)
    assert np.all((np.abs(got - ref) <= bound)[ok])
    assert np.all(np.abs(gl - rl)[ok] <= 1e-4)
    if where == "v":
        assert not np.isfinite(got[~ok][:, 3]).any()
        # the other columns do not mix with column 3
        cols = np.arange(128) != 3
        assert np.all((np.abs(got - ref) <= bound)[~ok][:, cols])
    elif np.isnan(bad):
        assert np.isnan(got[~ok]).all()


def test_attention_rows_without_a_position(w):
    """A cache shorter than the new tokens, pages that are not there, lengths of zero."""
    a = Attn([(0, 20), (100, 1), (60, 40), (30, 1), (0, 1)], 8, 2, 128, 16, "bf16", seed=8)
    a.L[0] = 6            # the first 14 tokens come before the cache's first position
    a.table[1, :] = -1    # no page at all
    a.table[2, 2] = 1 << 20
    a.table[2, 4] = -7
    a.L[4] = 0
    out, lse = a.run(w)
    a.check(out, lse)
    assert (out[:14] == 0).all() and (lse[:14] == -np.inf).all() and (out[20] == 0).all() and (out[-1] == 0).all()
    a.L[3] = 10 ** 9      # longer than its table: counted as the table's room
    a.table[3, 0] = int(a.table[3, 0])
    out, lse = a.run(w, window=50)
    a.check(out, lse, window=50)


def test_attention_large_scores_and_equal_keys(w):
    a = Attn([(400, 1), (20, 90)], 8, 2, 128, 16, "bf16", seed=9, qscale=30.0)  # a softmax of nearly one position
    out, lse = a.run(w)
    ref, _, spread = serving.paged_attention(f64(a.q), f64(a.kc), f64(a.vc), a.table, a.q_start, a.L)
    # scores up to ~200: f32 sums of 128 products leave 128 * 2^-24 of sum |q k| scale, below 4e-3 in the exponent
    err = np.abs(f64(out) - ref)
    assert np.all(err <= (2.0 ** -9 + 8e-3) * (spread + np.abs(ref)))
    a.q[:] = 0                                                                   # the mean of the values
    a.check(*a.run(w))


def test_attention_deterministic_streams_and_workspace(w):
    """Twice the same bits, on another stream, and with a GEMM's workspace whose counters stay at zero."""
    for lens in ([(3000, 1), (50, 1)], [(900, 130), (10, 1), (77, 16)]):
        a = Attn(lens, 8, 2, 128, 16, "bf16", seed=10)
        need = w.w4a16_paged_attention_workspace_bytes(a.q.shape[0], len(lens), 8, 2, 128, int(a.n.max()))
        ws = w.new_workspace(max(need, 1 << 17))
        first, l1 = a.run(w, workspace=ws)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        again, l2 = a.run(w, workspace=ws, stream=s, flags=0)
        s.synchronize()
        assert torch.equal(first, again) and torch.equal(l1, l2)
        assert ws[:65536].view(torch.int32).abs().sum().item() == 0
    if need:
        with pytest.raises(w.W4A16Error) as e:
            a.run(w, workspace=ws[:1024])
        assert e.value.status == w.W4A16_EWORKSPACE


def test_attention_offsets_past_32_bits(w):
    """Pages whose byte and element offsets do not fit 32 bits (5 GB of keys, 5 GB of values)."""
    page, Hkv, d = 256, 8, 128
    pages = (5 << 30) // (page * Hkv * d * 2) + 1
    kc = torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    for new in (1, 40):
        a = Attn([(300, new)], 16, 8, 128, page, "bf16", seed=11)
        moved = {int(p): pages - 1 - 2 * i for i, p in enumerate(a.table[0, :2])}
        table = a.table.copy()
        flat = torch.arange(300 + new, device="cuda")
        slots = i32(np.array([moved[int(a.table[0, j // page])] * page + j % page for j in range(300 + new)]))
        k, v = (c[torch.from_numpy(a.table[0]).cuda()[flat // page], :, flat % page] for c in (a.kc, a.vc))
        w.w4a16_kv_write(k.contiguous(), v.contiguous(), slots, kc, vc)
        for c, p in enumerate(a.table[0, :2]):
            table[0, c] = moved[int(p)]
        small_k, small_v, small_t = a.kc, a.vc, a.table
        a.kc, a.vc, a.table = kc, vc, table
        out, lse = a.run(w)
        a.table = small_t
        a.check(out, lse, kc=small_k, vc=small_v)


def test_attention_python_refusals(w):
    a = Attn([(20, 1)], 8, 2, 128, 16, "bf16")
    t, qs, L = i32(a.table), i32(a.q_start), i32(a.L)
    ok = lambda **k: w.w4a16_paged_attention(**{**dict(q=a.q, k_cache=a.kc, v_cache=a.vc, block_table=t, q_start=qs,  # noqa: E731
                                                       kv_len=L, max_q=1), **k})
    ok()
    for bad in (dict(q=a.q.float()), dict(q=a.q.cpu()), dict(k_cache=a.kc[0]), dict(v_cache=a.vc[:1]),
                dict(k_cache=a.kc.half()), dict(block_table=t.long()), dict(q_start=qs[:1]), dict(kv_len=L.long()),
                dict(out=torch.empty(1, 8, 64, dtype=a.dt, device="cuda")), dict(lse=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            ok(**bad)
    with pytest.raises(w.W4A16Error):
        ok(out=a.q)


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

def draw_rows(R, V, dtype, seed, sigma=2.2, head=14.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((R, V)) * sigma + head * r.random((R, V)) ** 64
    return torch.from_numpy(x).cuda().to(dtype), torch.from_numpy(r.exponential(size=(R, V)).astype(np.float32)).cuda()


def check_sample(w, x, e, t=None, k=None, p=None, m=None):
    dev = lambda a, dt: None if a is None else torch.tensor(np.asarray(a), dtype=dt, device="cuda")  # noqa: E731
    lp = torch.empty(x.shape[0], device="cuda")
    tok = w.w4a16_sample(x, e, dev(t, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(m, torch.float32),
                         logprob=lp)
    xs, es, tok, lp = x.float().cpu().numpy(), e.cpu().numpy(), tok.cpu().numpy(), lp.cpu().numpy()
    for i in range(len(xs)):
        ti, ki, pi, mi = (None if a is None else a[i] for a in (t, k, p, m))
        want, wl = serving.sample(xs[i], es[i], ti, ki, pi, mi)
        assert tok[i] == want, (i, ti, ki, pi, mi, tok[i], want)
        if np.isfinite(wl):
            assert abs(lp[i] - wl) <= 2e-5 + 2e-6 * abs(wl), (i, lp[i], wl)
        else:
            assert lp[i] == wl


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 50001, 151936])
def test_sample_filters_alone_and_together(w, V, dtype):
    R = 6 if V > 5000 else 12
    r = np.random.default_rng(V)
    x, e = draw_rows(R, V, dtype, V + 1)
    t = r.uniform(0.4, 1.5, R).astype(np.float32)
    t[0] = 0.0
    k = np.array([1, 2, 50, 0, 1000, V, V + 5, -1, 7, 3, 20, 40][:R])
    p = r.uniform(0.3, 0.99, R).astype(np.float32)
    m = np.exp(r.uniform(-6, -1, R)).astype(np.float32)
    check_sample(w, x, e)
    check_sample(w, x, e, t)
    check_sample(w, x, e, t, k=k)
    check_sample(w, x, e, t, p=p)
    check_sample(w, x, e, t, m=m)
    check_sample(w, x, e, t, k=k, p=p, m=m)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sample_flat_rows_and_ties(w, dtype):
    """Nuclei of tens of thousands of tokens, and rows whose logits are mostly equal."""
    V = 40000
    x, e = draw_rows(4, V, dtype, 5, sigma=0.5, head=0.0)
    check_sample(w, x, e, p=np.array([0.5, 0.9, 0.999, 0.01], np.float32))
    check_sample(w, x, e, k=np.array([30000, 5000, 39999, 2500]), p=np.array([0.97, 0.5, 0.9999, 0.99], np.float32))
    x[:] = 1.5
    x[1, 7::3] = 1.25
    x[2, 100] = 9.0
    x[3, :] = -2.0
    x[3, 39990:] = 3.0
    check_sample(w, x, e, k=np.array([17, 30001, 20000, 12]))
    # equal weights: the nucleus ends inside them; away from a boundary by a third of a weight
    check_sample(w, x[:1], e[:1], p=np.array([(12345 + 1 / 3) / V], np.float32))
    check_sample(w, x, e, k=np.array([17, 30001, 20000, 12]), m=np.array([0.5, 0.9, 0.001, 0.5], np.float32))


def test_sample_odd_rows(w):
    """-inf, NaN and infinite logits, masked rows, rows in a wider array, one row of noise for all."""
    V = 3001
    x, e = draw_rows(10, V + 3, torch.float32, 9)
    x, e = x[:, 1:V + 1], e[:1, 2:V + 2].expand(10, V)
    x[0, :] = -np.inf
    x[1, 5:] = -np.inf
    x[2, ::2] = np.nan
    x[3, :] = np.nan
    x[4, 17] = -np.inf
    x[5, 1:] = -np.inf
    big = np.array([0.7] * 10, np.float32)
    check_sample(w, x, e, big)
    check_sample(w, x, e, big, k=np.full(10, 9), p=np.full(10, 0.9, np.float32))
    check_sample(w, x, e, np.zeros(10, np.float32))
    x[6, 100] = np.inf
    tok = w.w4a16_sample(x, e, top_k=i32(np.full(10, 9)))
    assert tok[6].item() == 100
    # filters at and past their ends
    check_sample(w, x[7:], e[7:], p=np.array([0.0, -1.0, 1.0], np.float32), m=np.array([1.0, 2.0, -1.0], np.float32))
    # a tiny temperature: the largest logit wins whatever the noise
    tok = w.w4a16_sample(x[7:8], e[7:8], torch.tensor([1e-30], device="cuda"))
    assert tok.item() == int(x[7].argmax())


def test_sample_probabilities(w):
    """Draws with fresh noise follow the filtered, renormalised probabilities (chi-square over 8 kept tokens)."""
    V, n = 600, 4000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(V, device="cuda", generator=g) * 2
    e = torch.empty(n, V, device="cuda").exponential_(generator=g)
    k = i32(np.full(n, 8))
    tok = w.w4a16_sample(x.expand(n, V), e, top_k=k)
    top = torch.topk(x, 8)
    want = torch.softmax(top.values, 0).cpu().numpy() * n
    got = np.array([(tok == i).sum().item() for i in top.indices])
    assert got.sum() == n
    assert ((got - want) ** 2 / want).sum() < 29.9  # chi-square, 7 degrees of freedom: exceeded once in 10^4


def test_sample_python_refusals(w):
    x, e = draw_rows(3, 100, torch.float32, 1)
    for bad in (dict(logits=x.double()), dict(noise=e.half()), dict(noise=e[:2]), dict(top_k=i32([1, 2])),
                dict(temperature=torch.ones(3)), dict(top_p=torch.ones(3, device="cuda").half()),
                dict(logits=x.t()), dict(token=torch.empty(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises(ValueError):
            w.w4a16_sample(**{**dict(logits=x, noise=e), **bad})


def test_operators_count_their_launches(w):
    a = Attn([(20, 1)], 8, 2, 128, 16, "bf16")
    x, e = draw_rows(1, 100, torch.float32, 1)
    for f, least in ((lambda: a.run(w), 1), (lambda: w.w4a16_sample(x, e), 1),
                     (lambda: w.w4a16_kv_write(a.kc[0].transpose(0, 1), a.vc[0].transpose(0, 1).contiguous(), i32(np.full(16, -1)),
                                               a.kc.clone(), a.vc.clone()), 1),
                     (lambda: w.w4a16_page_plan(i32([3]), i32([1]), i32([5]), i32([[0, 0]]), 16, max_tokens=1), 1)):
        n0 = w.w4a16_launch_count()
        f()
        assert w.w4a16_launch_count() >= n0 + least


def test_workspaces_of_streams_and_graphs(w):
    """Calls without a workspace: two streams at once, a graph captured before and kept over a larger call."""
    def call_of(a):
        tables = i32(a.table), i32(a.q_start), i32(a.L)
        outs = [torch.zeros_like(a.q) for _ in range(5)]
        return outs, lambda i, **kw: w.w4a16_paged_attention(a.q, a.kc, a.vc, *tables, int(a.n.max()), out=outs[i], **kw)

    souts, small = call_of(Attn([(2000, 1), (50, 1)], 8, 2, 128, 16, "bf16", seed=21))
    louts, large = call_of(Attn([(2500, 1)] * 6 + [(700, 200)], 16, 4, 128, 16, "bf16", seed=22))
    small(0)
    large(0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for i in range(1, 5):
        small(i, stream=s1)
        large(i, stream=s2)
    torch.cuda.synchronize()
    for i in range(1, 5):
        assert torch.equal(souts[0], souts[i]) and torch.equal(louts[0], louts[i])
    for warm in (False, True):
        s = torch.cuda.Stream()
        if warm:
            small(1, stream=s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            small(1)
        large(1, stream=s)  # a larger workspace on the stream of the capture
        for _ in range(3):
            torch.cuda.synchronize()
            souts[1].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(souts[0], souts[1]) and torch.equal(louts[0], louts[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [9001, 60000])
def test_sample_cuts_to_the_token(w, V, dtype):
    """Random numbers by which the least of the kept tokens wins: the cut itself, for nuclei and k from a few to thousands."""
    R = 24
    r = np.random.default_rng(V)
    x, _ = draw_rows(R, V, dtype, V + 3)
    t = np.linspace(0.5, 1.6, R).astype(np.float32)
    z = (x.float().cpu().numpy() / t[:, None]).astype(np.float32)
    e = np.exp(1.5 * (z - z.max(1, keepdims=True)).astype(np.float64)).astype(np.float32)  # score: falls as z rises
    p = r.uniform(0.5, 0.995, R).astype(np.float32)
    k = np.unique(np.geomspace(2, min(V - 1, 6000), R).astype(int))
    k = np.concatenate([k, np.full(R - len(k), 777)])
    m = np.full(R, 1e-3, np.float32)
    dev = lambda a, dt=torch.float32: torch.tensor(a, dtype=dt, device="cuda")  # noqa: E731
    for ks, ps, ms in ((None, p, None), (k, None, None), (None, p, m), (k, p, None)):
        tok = w.w4a16_sample(x, dev(e), dev(t), None if ks is None else dev(ks, torch.int32),
                             None if ps is None else dev(ps), None if ms is None else dev(ms)).cpu().numpy()
        for i in range(R):
            order = np.lexsort((np.arange(V), -z[i].astype(np.float64)))
            zs = z[i][order].astype(np.float64)
            wt = np.exp(zs - zs[0])
            n = V if ks is None else min(V, int(ks[i]))
            ends = {n}
            if ps is not None:
                # a token is kept while the weight before it is below p of the total; sums in f32 and of up to
                # 8192 weights rounded to 2^-31 of the total are off by less than 2^-17 of it
                before, want = np.cumsum(wt[:n]) - wt[:n], float(ps[i]) * wt[:n].sum()
                eps = 2.0 ** -17 * wt[:n].sum()
                ends = set(range(max(1, int((before < want - eps).sum())), max(1, int((before < want + eps).sum())) + 1))
            if ms is not None:
                ends = {min(j, int((zs - zs[0] >= np.log(np.float64(ms[i])) - 2e-6).sum())) for j in ends} | \
                       {min(j, int((zs - zs[0] >= np.log(np.float64(ms[i])) + 2e-6).sum())) for j in ends}
            # of equal z the first kept one has the score of all
            allowed = {int(order[:j][zs[:j] == zs[j - 1]][0]) for j in ends}
            assert tok[i] in allowed, (i, float(t[i]), ks is not None and int(ks[i]), ps is not None and float(ps[i]),
                                       int(tok[i]), sorted(allowed)[:5], min(ends), max(ends))


def test_sample_cut_among_equals(w):
    """Cuts that fall into thousands of equal logits, above and below other tokens."""
    V, R = 30000, 6
    x = torch.full((R, V), -4.0, device="cuda")
    x[:, 100:9100] = 2.0           # 9000 equals: more than a list holds
    x[1:, 100:4000] = 3.0          # 3900 of them above the rest
    x[:, 20000:20040] = 6.0
    x[5, :] = 0.0
    e = torch.rand((R, V), generator=torch.Generator("cuda").manual_seed(1), device="cuda") + 0.5
    for k in ([41] * R, [3000] * R, [3941] * R, [9041] * R, [1, 40, 2048, 2049, 8193, 12345]):
        check_sample(w, x, e, k=np.array(k))
    for p in ([0.3] * R, [0.8] * R, [0.05, 0.1, 0.2, 0.5, 0.9, 0.25]):
        check_sample(w, x, e, p=np.array(p, np.float32))
        check_sample(w, x, e, p=np.array(p, np.float32), k=np.array([5000] * R))
