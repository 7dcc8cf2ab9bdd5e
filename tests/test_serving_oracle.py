"""Pins of the paged-serving oracle (oracle/serving.py) against facts the
definitions fix, and the host checks of the serving entry points (no GPU)."""
import ctypes
import os
import shutil

import numpy as np
import pytest

from oracle import serving


def test_plan_hand_worked():
    table = [[7, -5, -5, -5], [-5, -5, -5, -5], [3, 4, -5, -5]]
    # pages of 8: 5+4 tokens end in page 1, 0+8 fill one page, 16+0 need nothing
    t, qs, kv, pos, slots, used = serving.page_plan([5, 0, 16], [4, 8, 0], [20, 21, 22], table, 8, 14)
    assert t.tolist() == [[7, 20, -1, -1], [21, -1, -1, -1], [3, 4, -1, -1]]
    assert qs.tolist() == [0, 4, 12, 12] and kv.tolist() == [9, 8, 16] and used == 2
    assert pos.tolist() == [5, 6, 7, 8] + list(range(8)) + [-1, -1]
    assert slots.tolist() == [61, 62, 63, 160] + list(range(168, 176)) + [-1, -1]


def test_plan_runs_out_of_pages():
    t, _, _, _, slots, used = serving.page_plan([0, 0], [8, 9], [5], [[0, 0], [0, 0]], 8, 17)
    assert t.tolist() == [[5, -1], [-1, -1]] and used == 3
    assert slots.tolist() == list(range(40, 48)) + [-1] * 9


def test_attention_equals_dense_softmax():
    r = np.random.default_rng(0)
    pages, Hkv, page, d, Hq = 6, 2, 8, 16, 6
    kc, vc = r.standard_normal((2, pages, Hkv, page, d))
    table = np.array([[4, 1, 0], [5, 2, 3]])
    q = r.standard_normal((5, Hq, d))
    out, lse, _ = serving.paged_attention(q, kc, vc, table, [0, 3, 5], [19, 9])
    k0 = np.concatenate([kc[4], kc[1], kc[0]], axis=1)[:, :19]
    v0 = np.concatenate([vc[4], vc[1], vc[0]], axis=1)[:, :19]
    for i in range(3):
        for h in range(Hq):
            s = k0[h // 3, :17 + i] @ q[i, h] / 4.0
            w = np.exp(s)
            assert np.allclose(out[i, h], w @ v0[h // 3, :17 + i] / w.sum(), atol=1e-12)
            assert np.isclose(lse[i, h], np.log(w.sum()))
    # a window of one position returns that position's value; the block form sees the last one
    one, _, _ = serving.paged_attention(q, kc, vc, table, [0, 3, 5], [19, 9], window=1)
    assert np.allclose(one[4, 5], vc[2, 1, 0])
    blk, _, _ = serving.paged_attention(q, kc, vc, table, [0, 3, 5], [19, 9], window=1, block=True)
    assert np.allclose(blk[0, 0], vc[0, 0, 2])
    # pages that are not there, and tokens before the cache's first position
    gone, glse, _ = serving.paged_attention(q, kc, vc, np.array([[4, -1, 0], [9, 9, 9]]), [0, 3, 5], [2, 9])
    assert np.all(gone[0] == 0) and np.all(glse[0] == -np.inf) and np.all(gone[3:] == 0)
    assert np.allclose(gone[1, 0], vc[4, 0, 0])


def test_sample_filters():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.05, 0.25], dtype=np.float64)).astype(np.float32)
    e = np.array([1.0, 1.0, 1.0, 1e-9, 1.0], dtype=np.float32)  # token 3 wins wherever it is kept
    assert serving.sample(x, e)[0] == 3
    assert serving.sample(x, e, top_k=4)[0] == 1
    assert serving.sample(x, e, top_p=0.94)[0] == 1   # 0.4 + 0.25 + 0.2 + 0.1 reach it
    assert serving.sample(x, e, top_p=0.96)[0] == 3
    assert serving.sample(x, e, min_p=0.2)[0] == 1
    assert serving.sample(x, e, temperature=0.0)[0] == 1
    # top_p counts within what top_k left: 0.4 / 0.65 alone reaches 0.6, not 0.62
    e = np.array([1.0, 1.0, 1.0, 1.0, 1e-9], dtype=np.float32)
    assert serving.sample(x, e, top_k=2, top_p=0.6)[0] == 1
    assert serving.sample(x, e, top_k=2, top_p=0.62)[0] == 4
    # equal logits: the lower index stays
    assert serving.sample(np.zeros(4, np.float32), np.array([1, 1e-3, 1e-6, 1e-9], np.float32), top_k=2)[0] == 1
    tok, lp = serving.sample(x, e, top_k=1)
    assert tok == 1 and abs(lp - np.log(0.4)) < 1e-6
    assert serving.sample(np.full(3, -np.inf, np.float32), np.ones(3, np.float32)) == (-1, -np.inf)


def test_sample_race_draws_the_probabilities():
    r = np.random.default_rng(1)
    x = np.log(np.array([0.5, 0.3, 0.15, 0.05])).astype(np.float32)
    n = 20000
    got = np.bincount([serving.sample(x, r.exponential(size=4).astype(np.float32), top_k=3)[0] for _ in range(n)],
                      minlength=4) / n
    want = np.array([0.5, 0.3, 0.15, 0.0]) / 0.95
    assert np.all(np.abs(got - want) <= 5 * np.sqrt(want * (1 - want) / n) + 1e-12)  # five standard deviations


# ---- host checks of the entry points ---------------------------------------

nvcc_missing = shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc")
PTR = [0x10000000 * (i + 1) for i in range(12)]  # distinct aligned fake addresses


@pytest.fixture(scope="module")
def w():
    if nvcc_missing:
        pytest.skip("nvcc not available")
    from int4_weight_only_gemm_gb300 import _build
    _build.build()
    import int4_weight_only_gemm_gb300 as w
    return w


def call(w, name, st, order, base, **change):
    """Packs the struct's fields in order, with changes, and calls the entry point."""
    f = dict(base)
    assert set(change) <= set(f)
    f.update(change)
    return getattr(w.load_library(), name)(st.pack(*[f[k] for k in order]), None)


def fields(text):
    return text.split()


def test_plan_refusals(w):
    order = fields("past new free table q_start kv_len pos slots used stride B F cols T page flags")
    base = dict(zip(order, PTR[:9] + [16, 4, 10, 16, 8, 16, 1]))
    do = lambda **c: call(w, "w4a16_page_plan", w._PLAN_ARGS, order, base, **c)  # noqa: E731
    for p in ("past", "new", "free", "table", "q_start", "kv_len", "pos", "slots", "used"):
        assert do(**{p: 0}) == w.W4A16_EINVAL, p
        assert do(**{p: base[p] + 2}) == w.W4A16_EALIGN, p
    assert do(B=-1) == do(F=-1) == do(cols=0) == do(T=-1) == do(stride=15) == do(page=0) == w.W4A16_EINVAL
    assert do(flags=2) == w.W4A16_EINVAL
    assert do(page=24) == do(page=512) == do(page=4) == do(B=16385) == w.W4A16_EUNSUPPORTED
    assert do(slots=base["pos"] + 16) == w.W4A16_EINVAL       # outputs overlapping
    assert do(kv_len=base["past"]) == w.W4A16_EINVAL          # an output over an input
    assert w.load_library().w4a16_page_plan(None, None) == w.W4A16_EINVAL


def test_write_refusals(w):
    order = fields("k v slots kc vc kt kh vt vh kcp kch kcs vcp vch vcs T H d pages page dtype flags reserved")
    base = dict(zip(order, PTR[:5] + [256, 128, 256, 128, 4096, 2048, 128, 4096, 2048, 128, 8, 2, 128, 64, 16, 0, 1, 0]))
    do = lambda **c: call(w, "w4a16_kv_write", w._WRITE_ARGS, order, base, **c)  # noqa: E731
    for p in ("k", "v", "kc", "vc", "slots"):
        assert do(**{p: 0}) == w.W4A16_EINVAL, p
    for p in ("k", "v", "kc", "vc"):
        assert do(**{p: base[p] + 8}) == w.W4A16_EALIGN, p
    assert do(slots=base["slots"] + 1) == w.W4A16_EALIGN
    for s in ("kt", "kh", "vt", "vh", "kcp", "kch", "kcs", "vcp", "vch", "vcs"):
        assert do(**{s: base[s] + 4}) == w.W4A16_EALIGN, s
        assert do(**{s: -8}) == w.W4A16_EINVAL, s
    assert do(T=-1) == do(H=0) == do(d=0) == do(pages=0) == do(page=0) == do(reserved=1) == w.W4A16_EINVAL
    assert do(d=12) == do(d=2048) == do(page=20) == do(dtype=2) == do(pages=1 << 27) == w.W4A16_EUNSUPPORTED
    assert do(kc=base["k"] + 256) == w.W4A16_EINVAL           # cache over the source
    assert do(flags=4) == w.W4A16_EINVAL
    assert do(T=0, k=0, v=0, slots=0, kc=0, vc=0) == 0        # nothing to write: no pointer is read


ATTN = fields("q kc vc table q_start kv_len out lse ws ws_bytes qt qh ot oh kcp kch kcs vcp vch vcs stride "
              "T B Hq Hkv d pages page cols max_q window block dtype scale flags")


def attn_base():
    return dict(zip(ATTN, PTR[:9] + [1 << 27, 1024, 128, 1024, 128, 4096, 2048, 128, 4096, 2048, 128, 16,
                                     4, 2, 8, 2, 128, 64, 16, 16, 2, 0, 0, 0, 0.0, 1]))


def test_attention_refusals(w):
    do = lambda **c: call(w, "w4a16_paged_attention", w._ATTN_ARGS, ATTN, attn_base(), **c)  # noqa: E731
    base = attn_base()
    for p in ("q", "kc", "vc", "table", "q_start", "kv_len", "out"):
        assert do(**{p: 0}) == w.W4A16_EINVAL, p
    for p in ("q", "kc", "vc", "out"):
        assert do(**{p: base[p] + 8}) == w.W4A16_EALIGN, p
    for p in ("table", "q_start", "kv_len", "lse"):
        assert do(**{p: base[p] + 2}) == w.W4A16_EALIGN, p
    for s in ("qt", "qh", "ot", "oh", "kcp", "kch", "kcs", "vcp", "vch", "vcs"):
        assert do(**{s: base[s] + 4}) == w.W4A16_EALIGN, s
        assert do(**{s: -8}) == w.W4A16_EINVAL, s
    assert do(d=96) == do(d=256) == do(dtype=2) == do(page=48) == do(Hq=130) == w.W4A16_EUNSUPPORTED
    assert do(Hq=7) == do(Hkv=0) == do(T=-1) == do(B=-1) == do(max_q=-1) == do(pages=0) == w.W4A16_EINVAL
    assert do(cols=0) == do(stride=15) == do(window=-1) == do(block=2) == do(flags=8) == w.W4A16_EINVAL
    assert do(scale=float("nan")) == w.W4A16_EINVAL
    assert do(out=base["q"]) == do(lse=base["kc"]) == do(lse=base["out"]) == w.W4A16_EINVAL
    for none in (dict(T=0), dict(B=0), dict(max_q=0)):
        assert do(**none) == 0                                 # no new token: nothing is launched


def test_sample_refusals(w):
    order = fields("logits noise temperature top_k top_p min_p token logprob ws ws_bytes lrow nrow R V dtype flags")
    base = dict(zip(order, PTR[:9] + [1 << 20, 1000, 1000, 4, 1000, 0, 1]))
    do = lambda **c: call(w, "w4a16_sample", w._SAMPLE_ARGS, order, base, **c)  # noqa: E731
    for p in ("logits", "noise", "token"):
        assert do(**{p: 0}) == w.W4A16_EINVAL, p
    assert do(logits=base["logits"] + 1) == do(noise=base["noise"] + 2) == do(top_k=base["top_k"] + 1) == w.W4A16_EALIGN
    assert do(logits=base["logits"] + 2, dtype=2) == w.W4A16_EALIGN
    assert do(R=-1) == do(V=0) == do(lrow=-1) == do(nrow=-1) == do(flags=2) == w.W4A16_EINVAL
    assert do(dtype=3) == do(V=(1 << 24) + 1) == do(R=65536) == w.W4A16_EUNSUPPORTED
    assert do(token=base["logits"] + 16) == do(logprob=base["token"]) == w.W4A16_EINVAL
    assert do(R=0, logits=0, noise=0, token=0) == 0


def test_argument_structs_have_the_headers_sizes(w):
    assert [s.size for s in (w._PLAN_ARGS, w._WRITE_ARGS, w._ATTN_ARGS, w._SAMPLE_ARGS)] == [104, 152, 224, 112]
    for s in (w._PLAN_ARGS, w._WRITE_ARGS, w._ATTN_ARGS, w._SAMPLE_ARGS):
        assert s.size % ctypes.sizeof(ctypes.c_void_p) == 0
