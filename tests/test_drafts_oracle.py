"""Pins of the oracle of rotary positions, the 8-bit cache and tree attention (oracle/drafts.py), and the host checks
of their entry points (no GPU)."""
import ctypes
import math

import numpy as np
import pytest

import int4_weight_only_gemm_gb300 as w
from oracle import drafts, serving
from test_serving_oracle import ATTN, PTR, attn_base, call, fields


@pytest.fixture(scope="module", autouse=True)
def built():
    from int4_weight_only_gemm_gb300 import _build
    _build.build()


# ---------------------------------------------------------------------------
# the oracle
# ---------------------------------------------------------------------------

def test_rotation_keeps_lengths_and_depends_on_distance():
    r = np.random.default_rng(0)
    f, _ = drafts.frequencies(16)
    q, k = r.standard_normal((2, 1, 1, 20))
    for inter in (False, True):
        dots = []
        for p in (0, 7, 1000003):
            a, b = (drafts.rotate(x, [p + o], f, inter)[0, 0] for x, o in ((q, 5), (k, 0)))
            dots.append(a @ b)
            assert np.allclose(a[16:], q[0, 0, 16:]) and np.isclose(a @ a, q[0, 0] @ q[0, 0])
        assert np.allclose(dots, dots[0], atol=1e-9)
    # position 0 and negative ones leave the row, a quarter turn takes (1, 0) to (0, 1)
    assert np.array_equal(drafts.rotate(q, [0], f), q) and np.array_equal(drafts.rotate(q, [-1], f), q)
    x = np.zeros((1, 1, 4))
    x[0, 0, 0] = 1
    assert np.allclose(drafts.rotate(x, [1], [math.pi / 2, 0]), [[[0, 0, 1, 0]]])
    assert np.allclose(drafts.rotate(x, [1], [math.pi / 2, 0], True, 2.0), [[[0, 2, 0, 0]]])


def test_scalings_have_the_ends_they_are_made_for():
    plain, one = drafts.frequencies(64)
    assert one == 1 and plain[0] == 1 and np.isclose(plain[-1], 10000.0 ** (-62 / 64))
    base, _ = drafts.frequencies(64, scaling="base", factor=4)
    assert base[0] == 1 and np.isclose(base[-1], plain[-1] / 4)
    for s in ("ramp", "wavelength"):
        f, m = drafts.frequencies(64, scaling=s, factor=4, length=2048)
        turns = 2048 * plain / (2 * math.pi)
        assert np.allclose(f[turns > 40], plain[turns > 40]) and np.allclose(f[turns < 0.7], plain[turns < 0.7] / 4)
        assert np.all(f <= plain + 1e-15) and np.all(f >= plain / 4 - 1e-15)
        assert np.isclose(m, 0.1 * math.log(4) + 1 if s == "ramp" else 1)


@pytest.mark.parametrize("args", [(128,), (64, 500000.0, "linear", 4.0), (128, 10000.0, "base", 8.0), (2, 100.0, "base", 3.0),
                                  (64, 10000.0, "ramp", 8.0, 4096.0), (128, 1e6, "ramp", 40.0, 8192.0, 1.0, 4.0),
                                  (128, 500000.0, "wavelength", 8.0, 8192.0, 1.0, 4.0)])
def test_library_frequencies(args):
    """Computed on the host: f64 powers and logarithms differ by a few last places."""
    r, base, scaling, factor, length, low, high = (*args, 10000.0, "none", 1.0, 0.0, 1.0, 32.0)[:1] + \
        tuple(args[i] if len(args) > i else v for i, v in enumerate((None, 10000.0, "none", 1.0, 0.0, 1.0, 32.0)) if i)
    got, mag = w.w4a16_rope_frequencies(r, base, scaling, factor, length, low, high, device="cpu")
    want, m = drafts.frequencies(r, base, scaling, factor, length, low, high)
    assert np.allclose(got.numpy(), want, rtol=1e-14, atol=0) and abs(mag - m) <= 2.0 ** -23 * m


def test_e4m3_codes_and_their_values():
    torch = pytest.importorskip("torch")
    every = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    v = drafts.e4m3_value(every)
    assert np.array_equal(v, torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy())
    r = np.random.default_rng(1)
    x = np.concatenate([v, (v[1:] + v[:-1]) / 2, r.standard_normal(20000) * 100, r.standard_normal(20000) * 0.01])
    x = x[np.abs(x) <= 448].astype(np.float32)
    assert np.array_equal(drafts._e4m3_code(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("code,step", [("int8", 0.5 / 127), ("e4m3", None)])
def test_quantised_rows_are_within_half_a_step(code, step):
    r = np.random.default_rng(2)
    x = (r.standard_normal((50, 64)) * np.exp(r.uniform(-30, 30, (50, 1)))).astype(np.float32)
    codes, scale = drafts.quantise(x, code)
    amax = np.abs(x).max(-1, keepdims=True)
    # half a step of the grid (or of the code's own size, 2^-4, down to half the smallest code), and f32 roundings
    allowed = step * amax if step else np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * amax / 448)
    assert np.all(np.abs(drafts.values(codes, scale, code) - x) <= allowed * (1 + 1e-4) + amax * 2.0 ** -22)
    # the largest element of a row gets the largest code
    assert np.allclose(np.abs(drafts.values(codes, scale, code)).max(-1), amax[:, 0], rtol=2.0 ** -22)
    odd = np.zeros((4, 16), np.float32)
    odd[1, 3], odd[2, 5], odd[3, 0] = np.nan, -np.inf, 2.0 ** -101
    codes, scale = drafts.quantise(odd, code)
    assert not codes.any() and scale[0] == scale[3] == 0 and np.isnan(scale[1:3]).all()
    assert np.isnan(drafts.values(codes, scale, code)[1:3]).all()


def test_tree_attention_of_a_chain_is_causal_attention():
    r = np.random.default_rng(3)
    kc, vc = r.standard_normal((2, 6, 2, 8, 16))
    table, qs, kv = np.array([[4, 1, 0], [5, 2, 3]]), [0, 4, 9], [19, 9]
    q = r.standard_normal((9, 4, 16))
    chain = drafts.bits([range(i + 1) for i in range(4)] + [range(i + 1) for i in range(5)], 1)
    for window in (0, 3, 7):
        for a, b in zip(drafts.tree_attention(q, kc, vc, table, qs, kv, chain, window),
                        serving.paged_attention(q, kc, vc, table, qs, kv, window)):
            if window == 3:   # a path longer than the window is the caller's: it is seen whole
                a, b = a[[0, 1, 2, 4, 5, 6]], b[[0, 1, 2, 4, 5, 6]]
            assert np.allclose(a, b)
    # a star: each node sees the context and itself; a row without bits the context; no context and no bit: nothing
    star = drafts.bits([[0], [1], [], [3], [0], [1], [2], [3], []], 2)
    out, lse, _ = drafts.tree_attention(q, kc, vc, table, qs, [19, 5], star)
    one, _, _ = serving.paged_attention(q[1:2], kc, vc, np.array([[4, 1, 0]]), [0, 1], [15])
    assert np.isclose(lse[1, 0], np.logaddexp(
        np.log(np.sum(np.exp(np.concatenate([kc[4], kc[1]], 1)[0, :15] @ q[1, 0] / 4))), kc[0, 0, 0] @ q[1, 0] / 4))
    assert np.allclose(out[2], serving.paged_attention(q[2:3], kc, vc, np.array([[4, 1, 0]]), [0, 1], [15])[0][0])
    assert np.all(out[8] == 0) and np.all(lse[8] == -np.inf) and np.allclose(out[4, 3], vc[5, 1, 0])


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

A = [0x10000000 * (i + 1) for i in range(12)]
ROPE = fields("x out pos freq xt xh ot oh T heads d rot inter dtype magnitude flags")
STORE = fields("q k v q_out pos freq slots kc vc kscale vscale qt qh ot oh kt kh vt vh kcp kch kcs vcp vch vcs ksp ksh kss "
               "vsp vsh vss T Hq heads d rot inter pages page dtype code magnitude flags")
READ = fields("kc vc kscale vscale slots k v kt kh vt vh kcp kch kcs vcp vch vcs ksp ksh kss vsp vsh vss T heads d pages "
              "page dtype code flags")
EXT = fields("kscale vscale tree ksp ksh kss vsp vsh vss node code words")


def rope_base():
    return dict(zip(ROPE, A[:4] + [1024, 128, 1024, 128, 8, 8, 128, 128, 0, 0, 1.0, 1]))


def store_base():
    return dict(zip(STORE, A[:11] + [512, 128, 512, 128, 256, 128, 256, 128, 4096, 2048, 128, 4096, 2048, 128, 32, 16, 1,
                                     32, 16, 1, 8, 4, 2, 128, 128, 0, 64, 16, 0, 3, 1.0, 1]))


def read_base():
    return dict(zip(READ, A[:7] + [256, 128, 256, 128, 4096, 2048, 128, 4096, 2048, 128, 32, 16, 1, 32, 16, 1, 8, 2, 128,
                                   64, 16, 0, 3, 1]))


def refused(name, packer, order, base, cases):
    for status, changes in cases:
        for c in changes:
            assert call(w, name, packer, order, dict(base), **c) == status, (name, c)


def test_rope_refusals():
    E, L, U = w.W4A16_EINVAL, w.W4A16_EALIGN, w.W4A16_EUNSUPPORTED
    refused("w4a16_rope", w._ROPE_ARGS, ROPE, rope_base(), [
        (E, [dict(x=0), dict(out=0), dict(pos=0), dict(freq=0), dict(T=-1), dict(heads=0), dict(rot=0), dict(rot=7),
             dict(rot=130), dict(inter=2), dict(flags=2), dict(xt=-8), dict(ot=0), dict(oh=0), dict(d=0),
             dict(out=A[0] + 16), dict(out=A[0], oh=256), dict(pos=A[1] + 64), dict(freq=A[1] + 64)]),
        (L, [dict(x=A[0] + 2), dict(out=A[1] + 8), dict(pos=A[2] + 2), dict(freq=A[3] + 4), dict(xt=1020), dict(oh=132)]),
        (U, [dict(dtype=2), dict(dtype=3), dict(d=12, rot=8), dict(d=264), dict(heads=1025)]),
        (w.W4A16_OK, [dict(T=0)])])


def test_frequencies_refusals():
    lib = w.load_library()
    f, m = (ctypes.c_double * 64)(), ctypes.c_float()
    ok = dict(r=128, base=1e4, s=3, factor=8.0, length=4096.0, low=1.0, high=32.0)
    do = lambda **c: lib.w4a16_rope_frequencies(*{**ok, **c}.values(), f, ctypes.byref(m))  # noqa: E731
    assert do() == 0
    for c in (dict(r=0), dict(r=3), dict(r=-2), dict(base=0.0), dict(base=math.inf), dict(base=math.nan), dict(factor=0.0),
              dict(factor=math.nan), dict(s=5), dict(s=-1), dict(length=0.0), dict(low=32.0), dict(low=0.0), dict(high=math.inf)):
        assert do(**c) == w.W4A16_EINVAL, c
    assert do(s=0, length=0.0, low=0.0) == 0
    assert lib.w4a16_rope_frequencies(*ok.values(), None, ctypes.byref(m)) == w.W4A16_EINVAL
    with pytest.raises(ValueError):
        w.w4a16_rope_frequencies(64, scaling="other", device="cpu")
    for bad in (0, 7, -4):
        with pytest.raises(w.W4A16Error):
            w.w4a16_rope_frequencies(bad, device="cpu")


def test_store_refusals():
    E, L, U = w.W4A16_EINVAL, w.W4A16_EALIGN, w.W4A16_EUNSUPPORTED
    bare = dict(q=0, q_out=0, Hq=0, freq=0, pos=0, rot=0)
    refused("w4a16_kv_store", w._STORE_ARGS, STORE, store_base(), [
        (E, [dict(k=0), dict(v=0), dict(q=0), dict(q_out=0), dict(pos=0), dict(freq=0), dict(slots=0), dict(kc=0),
             dict(vc=0), dict(kscale=0), dict(vscale=0), dict(T=-1), dict(Hq=-1), dict(heads=0), dict(rot=0), dict(rot=9),
             dict(inter=3), dict(pages=0), dict(flags=4), dict(kcp=0), dict(vcs=0), dict(ksp=0), dict(vss=0), dict(ot=0),
             dict(kt=-8), dict(code=0), {**bare, "rot": 4}, {**bare, "Hq": 4},
             dict(kc=A[1]), dict(kscale=A[7]), dict(vscale=A[2]), dict(q_out=A[1]), dict(q_out=A[0] + 16), dict(q_out=A[9]),
             dict(slots=A[7])]),
        (L, [dict(k=A[1] + 2), dict(kc=A[7] + 8), dict(kscale=A[9] + 2), dict(freq=A[5] + 4), dict(kcs=136), dict(vch=2056),
             dict(kt=257), dict(q=A[0] + 4)]),
        (U, [dict(dtype=2), dict(code=1), dict(code=2), dict(code=5), dict(d=136, rot=8), dict(d=272), dict(page=24),
             dict(heads=1025), dict(pages=1 << 28)]),
        (w.W4A16_OK, [dict(T=0), {**bare, "T": 0}])])
    # 16-bit caches have no scales
    assert call(w, "w4a16_kv_store", w._STORE_ARGS, STORE, store_base(), code=0, kscale=0, vscale=0, T=0) == w.W4A16_OK
    # queries rotated in place beside the keys and values of the same rows
    fused = dict(q=A[0], q_out=A[0], k=A[0] + 1024, v=A[0] + 1536, qt=1024, ot=1024, kt=1024, vt=1024)
    for c in (dict(k=A[0] + 1008), dict(kt=1032), dict(v=A[0] + 512), dict(ot=2048)):
        assert call(w, "w4a16_kv_store", w._STORE_ARGS, STORE, store_base(), **{**fused, **c}) == E, c


def test_read_refusals():
    E, L, U = w.W4A16_EINVAL, w.W4A16_EALIGN, w.W4A16_EUNSUPPORTED
    refused("w4a16_kv_read", w._READ_ARGS, READ, read_base(), [
        (E, [dict(k=0), dict(v=0), dict(slots=0), dict(kc=0), dict(vc=0), dict(kscale=0), dict(T=-1), dict(heads=0),
             dict(pages=0), dict(flags=4), dict(kcp=0), dict(ksp=-1), dict(kt=0), dict(vh=0), dict(code=1, kscale=0, dtype=1),
             dict(k=A[0]), dict(v=A[3]), dict(k=A[6] + 64), dict(v=A[4])]),
        (L, [dict(k=A[5] + 2), dict(kc=A[0] + 8), dict(vscale=A[3] + 2), dict(kcs=136), dict(vt=257)]),
        (U, [dict(dtype=2), dict(code=0, dtype=1), dict(code=2), dict(d=136), dict(d=1040), dict(page=24), dict(heads=1025)]),
        (w.W4A16_OK, [dict(T=0)])])


def test_attention_extension_refusals():
    E, L, U = w.W4A16_EINVAL, w.W4A16_EALIGN, w.W4A16_EUNSUPPORTED
    lib = w.load_library()
    ext = dict(zip(EXT, [0x710000000, 0x720000000, 0x730000000, 32, 16, 1, 32, 16, 1, 2, 3, 2]))

    def do(args=(), **c):
        b = attn_base()
        b.update(dict(args))
        a = w._ATTN_ARGS.pack(*[b[k] for k in ATTN])
        x = {**ext, **c}
        return lib.w4a16_paged_attention_ex(a, w._EXT_ARGS.pack(*[x[k] for k in EXT]), None)

    for c in (dict(kscale=0), dict(vscale=0), dict(ksp=-1), dict(vss=-1), dict(words=0), dict(tree=0), dict(node=1),
              dict(code=0), dict(kscale=attn_base()["out"]), dict(tree=attn_base()["out"])):
        assert do(**c) == E, c
    # what is right comes as far as the workspace (or, without a GPU, the question for its size)
    late = (w.W4A16_EWORKSPACE, w.W4A16_ECUDA)
    assert do(dict(block=1)) == E and do(dict(block=1, ws=0), tree=0, words=0) in late
    for c in (dict(kscale=0x710000002), dict(tree=0x730000001)):
        assert do(**c) == L, c
    for s in ("kcp", "kch", "kcs", "vcp", "vch", "vcs"):
        assert do({s: 4096 + 8}) == L, s   # 16 elements of 8 bits
    for c in (dict(words=65, node=65), dict(code=2), dict(code=1), dict(code=5)):
        assert do(**c) == U, c
    none = dict(kscale=0, vscale=0, code=0)
    assert do(dict(ws=0), **none, tree=0, words=0) in late and do(dict(ws=0), **none) in late and do(dict(ws=0)) in late
