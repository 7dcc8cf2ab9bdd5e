"""Serving operators where their definitions are exact and floats are not: equal quotients of unequal logits, filters
wider than a masked row, lengths and windows near the ends of int32, long contexts with a NaN."""
import numpy as np
import pytest
import torch

from oracle import serving
from test_serving import Attn, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import int4_weight_only_gemm_gb300 as w
    return w


def dev(a, dtype=torch.float32):
    return None if a is None else torch.tensor(np.asarray(a), dtype=dtype, device="cuda")


def draws(w, x, e, t=None, k=None, p=None, m=None):
    """Tokens of the kernel and of the oracle; logits x and random numbers e are f32 arrays [R, V]."""
    logprob = torch.empty(len(x), device="cuda")
    token = w.w4a16_sample(dev(x), dev(e), dev(t), dev(k, torch.int32), dev(p), dev(m), logprob=logprob)
    of = lambda a, i: None if a is None else a[i]  # noqa: E731
    want = [serving.sample(x[i], e[i], of(t, i), of(k, i), of(p, i), of(m, i)) for i in range(len(x))]
    for got, (_, ref) in zip(logprob.tolist(), want):
        assert abs(got - ref) <= 2e-5 + 2e-6 * abs(ref)
    return token.tolist(), [a for a, _ in want]


# ---------------------------------------------------------------------------
# sampling: equal quotients of unequal logits
# ---------------------------------------------------------------------------

def step(x, n):
    """The f32 number n steps from x."""
    for _ in range(abs(n)):
        x = np.nextafter(np.float32(x), np.float32(np.inf if n > 0 else -np.inf))
    return np.float32(x)


def test_the_largest_quotient_at_the_lower_index(w):
    """l / 1.5 rounds two neighbouring logits to one quotient: of equal ones the lower index is first, whichever logit
    it has."""
    V, T = 40000, np.float32(1.5)
    tops = [a for a in (step(15.0, i) for i in range(64)) if np.float32(a) / T == np.float32(step(a, -1)) / T][:8]
    assert len(tops) == 8
    x = np.full((8, V), -4.0, np.float32)
    for i, a in enumerate(tops):
        x[i, 30000 + 3 * i] = a
        x[i, 11 + 997 * i] = step(a, -1)
    e = np.ones((8, V), np.float32)
    t = np.full(8, T, np.float32)
    first = [11 + 997 * i for i in range(8)]
    for more in (dict(k=np.ones(8, int)), dict(p=np.full(8, 1e-3, np.float32)), dict(k=np.ones(8, int), p=np.full(8, 0.5, np.float32))):
        got, want = draws(w, x, e, t, **more)
        assert want == first and got == want


@pytest.mark.parametrize("k", [5, 9, 13])
def test_pairs_of_one_load_with_one_quotient(w, k):
    """Pairs of neighbouring logits, one quotient for all: the first k of the row stay, not the larger of each pair."""
    V, T = 40000, np.float32(1.9)
    hi = np.float32(1.9500003)
    lo = step(hi, -1)
    assert lo / T == hi / T
    x = np.full((1, V), -4.0, np.float32)
    order = []
    for j in range(1, 11):
        x[0, 400 * j], x[0, 400 * j + 1] = lo, hi
        order += [400 * j, 400 * j + 1]
    for last in range(k):  # the one with the smallest random number is drawn if it is kept
        e = np.ones((1, V), np.float32)
        e[0, order[last]] = 1e-4
        got, want = draws(w, x, e, np.array([T]), k=np.array([k]))
        assert want == [order[last]] and got == want
    mass = np.exp(-4 / 1.9 - 1.9500003 / 1.9) * (V - 20) + 20
    p = np.array([(k - 0.5) / mass], np.float32)
    for last in range(k):
        e = np.ones((1, V), np.float32)
        e[0, order[last]] = 1e-4
        got, want = draws(w, x, e, np.array([T]), p=p)
        assert want == [order[last]] and got == want


def test_top_k_ends_where_counting_ends(w):
    """The k-th token forty units of z below the first, where the kernel stops counting tokens of a large k."""
    V, T, k, R = 40000, np.float32(1.5), 1500, 25
    x = np.full((R, V), -1000.0, np.float32)
    x[:, 1000:1000 + k - 1] = 10.0
    e = np.ones((R, V), np.float32)
    e[:, [3, 50]] = 1e-30
    equal = 0
    for i in range(R):
        x[i, 50] = step(np.float32(10.0) - np.float32(40.0) * T * np.float32(1.0001), i - R // 2)
        x[i, 3] = step(x[i, 50], -1)
        equal += x[i, 50] / T == x[i, 3] / T
    assert equal >= 5
    got, want = draws(w, x, e, np.full(R, T), k=np.full(R, k))
    assert got == want and want.count(3) == equal


# ---------------------------------------------------------------------------
# sampling: rows of which a mask leaves less than top-k
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("V", [1500, 3001, 40000, 151936])
def test_top_p_of_a_row_with_fewer_tokens_than_top_k(w, V):
    """Five tokens are left by a mask, top-k takes fifty (or 3000), top-p cuts among the five."""
    R = 6
    x = np.full((R, V), -np.inf, np.float32)
    at = np.array([7, 100, 101, V // 2, V - 1])
    x[:, at] = np.array([1.0, 3.0, 2.0, 2.5, -4.0])  # .064, .474, .174, .287 and .0004 of the probability
    e = np.ones((R, V), np.float32)
    for i in range(5):
        e[i, at[i]] = 1e-6   # drawn if it is kept
    p = np.array([0.3, 0.6, 0.6, 0.9, 0.9, 0.99], np.float32)
    for k in (50, 3000):
        for more in ({}, dict(m=np.full(R, 1e-6, np.float32))):
            got, want = draws(w, x, e, k=np.full(R, k), p=p, **more)
            assert got == want
            got, want = draws(w, x, e, k=np.full(R, k), p=p[::-1].copy(), **more)
            assert got == want


# ---------------------------------------------------------------------------
# plan: lengths and pages near the ends of int32
# ---------------------------------------------------------------------------

MOST = 2 ** 31 - 1


def plan(w, past, new, free, table, page, tokens):
    """-> table, q_start, kv_len, positions, slots, used as lists."""
    t = dev(table, torch.int32)
    out = w.w4a16_page_plan(dev(past, torch.int32), dev(new, torch.int32), dev(free, torch.int32), t, page,
                            max_tokens=tokens)
    return [t.tolist()] + [x.tolist() for x in out]


def test_plan_with_a_cache_as_long_as_int32(w):
    table, q_start, kv_len, positions, slots, used = plan(
        w, [MOST, 5, MOST - 4], [1, 3, 100], [40, 41], [[1, 2], [3, 4], [5, 6]], 16, 9)
    assert table == [[1, 2], [3, -1], [5, 6]]
    assert q_start == [0, 0, 3, 7] and kv_len == [MOST, 8, MOST]
    assert positions == [5, 6, 7] + [MOST - 4 + i for i in range(4)] + [-1, -1]
    assert slots == [53, 54, 55] + [-1] * 6 and used == [0]


@pytest.mark.parametrize("page", [8, 16, 256])
def test_plan_with_more_new_tokens_than_int32_holds(w, page):
    T, pages = 2 * page + 3, 2 ** 31 // page
    table, q_start, kv_len, positions, slots, used = plan(
        w, [0, 0, 3], [MOST, MOST, 7], [40, 41, 42, 43], [[1, 2, 3]] * 3, page, T)
    assert table == [[40, 41, 42], [-1] * 3, [1, -1, -1]]
    assert q_start == [0, MOST, MOST, MOST] and kv_len == [MOST, MOST, 10]
    assert positions == list(range(T))
    assert slots == [(40 + i // page) * page + i % page for i in range(T)]
    assert used == [2 * pages + (10 > page)]


def test_plan_whose_pages_sum_past_int32(w):
    B = 16384
    past = np.zeros(B, int)
    new = np.full(B, MOST)
    new[-1] = 0
    table, q_start, kv_len, positions, slots, used = plan(w, past, new, [7], np.zeros((B, 1), int), 8, 20)
    assert table == [[7]] + [[-1]] * (B - 1) and q_start == [0] + [MOST] * B and used == [MOST]
    assert kv_len == new.tolist() and positions == list(range(20)) and slots == list(range(56, 64)) + [-1] * 12


def test_plan_page_past_the_last_slot(w):
    """A page number whose slots do not fit int32 gives no slot, and none of another page."""
    last = 2 ** 31 // 16 - 1
    table, _, _, _, slots, _ = plan(w, [3, 3, 16], [1, 1, 1], [last + 1], [[last, 0], [2 ** 28, 0], [9, 0]], 16, 3)
    assert slots == [last * 16 + 3, -1, -1]
    assert table[2] == [9, last + 1]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3, 2 ** 30])
@pytest.mark.parametrize("new,L", [(4, 2), (4, 4), (20, 6), (150, 70)])
def test_window_as_large_as_it_gets(w, window, new, L):
    """No window in effect, also where the first tokens come before the cache's first position."""
    a = Attn([(0, new), (40, new)], 8, 2, 128, 16, "bf16", seed=12)
    a.L[0] = L
    out, lse = a.run(w, window)
    a.check(out, lse)
    free, _ = a.run(w, 0)
    assert torch.equal(out, free)


def spoil(a, spots):
    """Puts values that are not finite into the value cache: (request, position, column, value)."""
    for b, j, col, x in spots:
        a.vc[int(a.table[b, j // a.page]), a.Hkv - 1, j % a.page, col] = x


@pytest.mark.parametrize("heads", [(8, 2, 128, "bf16"), (4, 1, 64, "fp16"), (3, 3, 128, "fp16"), (64, 1, 64, "bf16")])
@pytest.mark.parametrize("lens,window", [([(700, 300)], 0), ([(70, 150), (200, 19)], 0), ([(0, 600)], 64),
                                         ([(1500, 200), (3, 1)], 5), ([(4000, 40)], 300), ([(0, 260), (900, 270)], 0)])
def test_values_that_some_tokens_of_a_chunk_see(w, heads, lens, window):
    """Infinities and NaN among the new tokens' own values: in the columns of the tokens that see them, nowhere else."""
    Hq, Hkv, d, dtype = heads
    a = Attn(lens, Hq, Hkv, d, 16, dtype, seed=13)
    r = np.random.default_rng(5)
    spots = []
    for b, (past, new) in enumerate(lens):
        for x in (np.nan, np.inf, -np.inf, np.inf, np.nan, -np.inf):
            spots.append((b, past + int(r.integers(0, new)), int(r.integers(0, d)), x))
        spots.append((b, past + new - 1, 0, np.inf))
        spots.append((b, past + new - 1, 1, -np.inf))
    spoil(a, spots)
    out, lse = a.run(w, window)
    assert w.w4a16_last_device_status() == 0
    a.check(out, lse, window)
    last = int(a.n[0]) - 1  # the newest token: its own infinities, with their signs
    got = f64(out)[last, -1]
    seen = {c for b, j, c, x in spots if b == 0 and c < 2 and j < lens[0][0] + lens[0][1] - 1}
    for c, want in ((0, np.inf), (1, -np.inf)):
        if c not in seen:
            assert got[c] == want


def test_a_nan_at_the_end_of_a_long_context(w):
    """What it costs does not grow with the context, and no wait of the kernel runs out over it."""
    past, new, page = 300000, 40, 256
    a = Attn([(past, new)], 2, 1, 64, page, "bf16", seed=14)
    spoil(a, [(0, past + 17, 5, np.nan), (0, past + 30, 6, np.inf)])
    a.run(w)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    out, lse = a.run(w)
    end.record()
    torch.cuda.synchronize()
    assert w.w4a16_last_device_status() == 0
    assert start.elapsed_time(end) < 100  # ms; every row anew takes seconds
    a.check(out, lse)
    bad = ~np.isfinite(f64(out))
    want = np.zeros_like(bad)
    want[17:, :, 5] = True
    want[30:, :, 6] = True
    assert np.array_equal(bad, want)


# ---------------------------------------------------------------------------
# sampling: temperatures near the ends of f32
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("V", [1500, 40000])
@pytest.mark.parametrize("positive", [False, True])
def test_temperatures_near_the_ends_of_f32(w, V, positive):
    t = np.array([1e-45, 1e-39, 1e-38, 1e-30, 1e30, 3e38, np.inf, np.nan], np.float32)
    R = len(t)
    r = np.random.default_rng(V)
    x = (r.standard_normal((R, V)) * 3 + (20 if positive else -40)).astype(np.float32)
    x[:, 5::11] = -np.inf
    e = r.exponential(size=(R, V)).astype(np.float32)
    as_if = np.where(np.isnan(t), np.float32(0), np.clip(t, np.float32(1e-30), np.float32(1e30)))
    for more in ({}, dict(k=np.full(R, 40)), dict(p=np.full(R, 0.5003, np.float32)), dict(m=np.full(R, 0.1, np.float32)),
                 dict(k=np.full(R, 3000), p=np.full(R, 0.9, np.float32), m=np.full(R, 0.01, np.float32))):
        want = [serving.sample(x[i], e[i], as_if[i], *(more[f][i] if f in more else None for f in "kpm")) for i in range(R)]
        lp = torch.empty(R, device="cuda")
        tok = w.w4a16_sample(dev(x), dev(e), dev(t), dev(more.get("k"), torch.int32), dev(more.get("p")),
                             dev(more.get("m")), logprob=lp)
        # (an infinite or equal draw apart: at 1e30 all quotients are below 1e-28 and the race is the noise's alone)
        assert tok.tolist() == [a for a, _ in want], more.keys()
        assert np.all(np.abs(lp.cpu().numpy() - [b for _, b in want]) <= 1e-4)
