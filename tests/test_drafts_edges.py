"""Rotary positions, the 8-bit cache and drafted trees where calls meet: captures and replays, streams side by side,
offsets past 32 bits, many requests, lengths at their ends.  Tolerances as in test_drafts.py."""
import numpy as np
import pytest
import torch

from oracle import drafts
from test_drafts import Draft, partner_sum
from test_serving import f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import int4_weight_only_gemm_gb300 as w
    return w


def step_of(w, a, seed, new):
    """Queries, keys and values of new tokens behind the requests' context, and the call that rotates, stores and attends."""
    g = torch.Generator("cuda").manual_seed(seed)
    T, d, Hkv = int(sum(new)), a.d, a.Hkv
    qkv = torch.randn(T, a.Hq + 2 * Hkv, d, generator=g, device="cuda").to(a.dt)
    positions = torch.cat([torch.arange(L - n, L) for L, n in zip(a.L.tolist(), new)])
    slots = torch.cat([torch.from_numpy(a.table[b])[torch.arange(L - n, L) // a.page] * a.page + torch.arange(L - n, L) % a.page
                       for b, (L, n) in enumerate(zip(a.L.tolist(), new))])
    f, _ = w.w4a16_rope_frequencies(d)
    st = dict(qkv=qkv, pos=i32(positions), slots=i32(slots), q=torch.empty_like(qkv[:, :a.Hq]).contiguous(),
              table=i32(a.table), start=i32(a.q_start), L=i32(a.L), out=torch.zeros(T, a.Hq, d, dtype=a.dt, device="cuda"))

    st["tree"] = None if a.tree is None else i32(a.tree)

    def call():
        q, k, v = st["qkv"].split([a.Hq, Hkv, Hkv], dim=1)
        scales = dict(k_scale=a.ks, v_scale=a.vs) if a.code else {}
        w.w4a16_rope_kv_write(q, k, v, st["pos"], f, st["slots"], a.kc, a.vc, q_out=st["q"], **scales)
        w.w4a16_paged_attention(st["q"], a.kc, a.vc, st["table"], st["start"], st["L"], int(max(new)), out=st["out"],
                                tree=st["tree"], **scales)
        return st["out"]

    return st, call


@pytest.mark.parametrize("code", [None, "int8", "e4m3"])
@pytest.mark.parametrize("lens,tree", [([(300, 1), (40, 1)], None), ([(200, 40), (9, 3)], None), ([(500, 3), (20, 2)], "tree"),
                                       ([(300, 70), (30, 40)], "tree")])
def test_captured_and_replayed_beside_eager_calls(w, code, lens, tree):
    a = Draft(lens, 8, 2, 128, 16, "bf16", code, tree, seed=1)
    st, call = step_of(w, a, 5, a.n)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (6, 7):
        st["qkv"].copy_(torch.randn(st["qkv"].shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda"))
        want = call().clone()
        state = [x.clone() for x in (a.kc.view(torch.uint8), a.vc.view(torch.uint8))]
        st["out"].zero_()
        graph.replay()
        assert torch.equal(st["out"], want)
        assert all(torch.equal(x, y.view(torch.uint8)) for x, y in zip(state, (a.kc, a.vc)))
    # replays beside calls of the same kind on another stream
    other = Draft(lens, 8, 2, 128, 16, "bf16", code, tree, seed=2)
    so, oc = step_of(w, other, 8, other.n)
    ref = oc().clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        graph.replay()
        with torch.cuda.stream(s):
            oc()
    torch.cuda.synchronize()
    assert torch.equal(so["out"], ref) and torch.equal(st["out"], want)
    assert w.w4a16_last_device_status() == 0


@pytest.mark.parametrize("lens,tree", [([(300, 1)], None), ([(250, 70)], None), ([(250, 3)], "tree"), ([(250, 70)], "tree")])
def test_offsets_past_32_bits(w, lens, tree):
    """A cache whose last pages lie more than 2^31 elements behind its first."""
    a = Draft(lens, 4, 2, 128, 128, "bf16", "int8", tree, seed=3)
    held = a.kc.shape[0]
    pages = 66000
    assert pages * 2 * 128 * 128 > 2 ** 31
    small = [a.kc, a.vc, a.ks, a.vs]
    big = [torch.zeros((pages,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in small]
    for x, y in zip(big, small):
        x[-held:] = y
    kc, vc, ks, vs = big
    out, lse = a.run(w)
    a.kc, a.vc, a.ks, a.vs = big
    a.table = np.where(a.table >= 0, a.table + pages - held, -1)
    again, lse2 = a.run(w)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # writing and reading there
    k = torch.randn(2, 5, 2, 128, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * 128 - 1 - i for i in range(5)], dtype=torch.int32, device="cuda")
    w.w4a16_kv_write(k[0], k[1], slots, kc, vc, k_scale=ks, v_scale=vs)
    back = torch.zeros_like(k)
    w.w4a16_kv_read(kc, vc, slots, back[0], back[1], k_scale=ks, v_scale=vs)
    codes, scale = drafts.quantise(k.float().cpu().numpy(), "int8")
    ref = drafts.values(codes, scale, "int8")
    assert np.all(np.abs(f64(back) - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref))
    assert not kc[0].any() and not vc[0].any() and not ks[0].any()


@pytest.mark.parametrize("code,tree", [("int8", None), ("e4m3", "tree"), (None, "tree"), ("int8", "any")])
def test_many_requests(w, code, tree):
    """More requests than a CTA has threads, most of them short, some without a token."""
    r = np.random.default_rng(4)
    lens = [(int(p), int(n)) for p, n in zip(r.integers(0, 40, 700), r.integers(0, 4, 700))]
    lens[350] = (900, 2)
    if tree is None:
        lens[20], lens[699] = (100, 40), (10, 60)
    a = Draft(lens, 4, 2, 64, 16, "bf16", code, tree, seed=5)
    a.check(*a.run(w))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("heads,kv_heads,lens", [(64, 1, [(33, 1), (200, 2)]), (9, 1, [(65, 1)]), (12, 12, [(10, 16), (7, 8)]),
                                                 (24, 3, [(129, 1), (128, 2)]), (16, 1, [(500, 1), (3, 1)])])
def test_rows_at_the_kernels_limits(w, code, heads, kv_heads, lens):
    """8, 9, 16 and more query rows a key head, in one call and alone."""
    for d, dtype in ((64, "fp16"), (128, "bf16")):
        a = Draft(lens, heads, kv_heads, d, 16, dtype, code, seed=6)
        a.check(*a.run(w))
        a.check(*a.run(w, 30), 30)


def test_all_zero_and_equal_scales(w):
    """Rows of zeros (scale 0) are values of zero, not of nothing."""
    for lens in ([(50, 1)], [(50, 40)]):
        a = Draft(lens, 8, 2, 128, 16, "bf16", "int8", seed=7)
        a.vs[:] = 0
        out, lse = a.run(w)
        a.check(out, lse)
        assert (out == 0).all() and torch.isfinite(lse).all()
        a.ks[:] = 0    # every score 0: the mean of the values
        a.vs[:] = 0.01
        a.check(*a.run(w))


def test_more_nodes_than_a_row_tile_and_the_widest_mask(w):
    """2048 nodes, the most that a mask has words for, as chains of chains; and masks wider than the tree."""
    n = 2048
    a = Draft([(20, n)], 1, 1, 64, 64, "bf16", None, "chain", seed=8)
    assert a.words == 64
    out, lse = a.run(w)
    b = Draft([(20, n)], 1, 1, 64, 64, "bf16", seed=8)
    b.check(out, lse)
    c = Draft([(40, 5), (3, 30)], 4, 2, 128, 16, "bf16", "int8", "tree", words=64, seed=9)
    c.check(*c.run(w))


def test_rope_in_place_on_a_side_stream(w):
    x = torch.randn(500, 12, 128, device="cuda").to(torch.bfloat16)
    kept = f64(x)
    pos = np.arange(500) * 37
    f, m = w.w4a16_rope_frequencies(128, scaling="ramp", factor=8.0, length=4096)
    positions = i32(pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w.w4a16_rope(x, positions, f, magnitude=m, out=x, stream=s)
    s.synchronize()
    ref = drafts.rotate(kept, pos, f64(f), False, m)
    assert np.all(np.abs(f64(x) - ref) <= m * 2.0 ** -21 * partner_sum(kept, 64, False) + 2.0 ** -8 * np.abs(ref))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("far", [0, 12, 20])
@pytest.mark.parametrize("lens,tree", [([(900, 130), (300, 70)], None), ([(700, 60), (280, 90)], "tree")])
def test_fp16_weights_of_long_rows(w, code, far, lens, tree):
    """Rows of 256 positions and more have weights of one part, 11 bits: rounded by 2^-11 of themselves or by 2^-25.  The base
    is at most the largest score + log2 (the largest scale, rounded up to a power of two) - 6, so that the key of the largest
    score has a weight of 2^5 / (largest scale) at least before its value's scale, and the row's sum is no less.  So
    |out - ref| <= (2^-11 + 2e-4) sum p|v| + 2^-11 |ref| + 2^-25 + n 2^-30 largest scale * 127 (or 480) with n positions.
    Some values are 2^far times larger."""
    a = Draft(lens, 8, 2, 128, 16, "fp16", code, tree, seed=11)
    a.vs *= 2.0 ** -10
    a.vs[torch.rand(a.vs.shape, generator=torch.Generator("cuda").manual_seed(1), device="cuda") < 0.02] *= 2.0 ** far
    out, lse = a.run(w)
    ref, rl, spread, _ = a.reference()
    most = float(a.vs.max()) * (127 if code == "int8" else 480)
    bound = (2.0 ** -11 + 2e-4) * spread + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + a.L.max() * 2.0 ** -30 * most
    assert np.all(np.abs(f64(out) - ref) <= bound)
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4 + 1e-6 * np.abs(rl))


@pytest.mark.parametrize("lens", [[(900, 130)], [(40, 50), (5, 9)], [(100, 1)]])
def test_fp16_rows_of_zeros_and_mixed_with_them(w, lens):
    a = Draft(lens, 8, 2, 128, 16, "fp16", "int8", seed=12)
    keep = a.vs.clone()
    a.vs[:] = 0
    out, lse = a.run(w)
    a.check(out, lse)
    assert (out == 0).all() and torch.isfinite(lse).all()
    a.vs[:] = torch.where(torch.rand(keep.shape, device="cuda") < 0.5, keep, torch.zeros_like(keep))
    ref, rl, spread, _ = a.reference()
    out, lse = a.run(w)
    assert np.all(np.abs(f64(out) - ref) <= (2.0 ** -11 + 2e-4) * spread + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4 + 1e-6 * np.abs(rl))


@pytest.mark.parametrize("code,tree", [("int8", None), ("e4m3", "tree"), ("e4m3", None)])
def test_few_rows_cut_over_many_ctas(w, code, tree):
    """Requests whose keys fall to many CTAs, next to requests of one CTA: a CTA that joins goes on with the next request."""
    for heads, kv_heads, d in ((4, 1, 128), (8, 2, 64), (6, 2, 128), (2, 2, 128)):
        lens = [(9000, 1), (40, 1), (3001, 1), (0, 1), (500, 1), (7011, 1), (130, 1)]
        a = Draft(lens, heads, kv_heads, d, 16, "bf16", code, tree, seed=31)
        a.check(*a.run(w))
        a.check(*a.run(w, 2000), 2000)
        b = Draft([(2303, 1)], heads, kv_heads, d, 64, "fp16", code, tree, seed=32)
        b.check(*b.run(w))


def test_tensors_of_another_device_are_refused(w, monkeypatch):
    a = Draft([(20, 2)], 4, 2, 64, 16, "bf16", "int8", seed=33)
    f, _ = w.w4a16_rope_frequencies(64)
    T = a.q.shape[0]
    at, k = i32(np.zeros(T)), torch.zeros(T, 2, 64, dtype=a.dt, device="cuda")
    before = a.kc.clone()
    calls = [lambda: w.w4a16_rope(a.q, at, f), lambda: a.run(w),
             lambda: w.w4a16_kv_write(k, k, at, a.kc, a.vc, k_scale=a.ks, v_scale=a.vs),
             lambda: w.w4a16_rope_kv_write(None, k, k, at, f, at, a.kc, a.vc, k_scale=a.ks, v_scale=a.vs),
             lambda: w.w4a16_kv_read(a.kc, a.vc, at, k, k.clone(), a.ks, a.vs)]
    for call in calls:
        with monkeypatch.context() as m:
            m.setattr(w, "_current", lambda: 1)   # as with torch.cuda.device(1) around the call
            with pytest.raises(ValueError, match="device"):
                call()
    with pytest.raises(ValueError):
        w.w4a16_kv_write(k, k, at, None, None)
    torch.cuda.synchronize()
    assert torch.equal(a.kc, before)
