"""Attention over an 8-bit cache in fp16 with more than 16 query rows a key head: its weights are taken against a base that
the values' scales are part of, and neither the softmax's sum nor the outputs may depend on how these scales run."""
import math

import numpy as np
import pytest
import torch

from test_drafts import Draft
from test_serving import f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import int4_weight_only_gemm_gb300 as w
    return w


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("small,large", [(0.0, 2.0 ** 40), (0.0, 2.0 ** 100), (2.0 ** -60, 2.0 ** 70), (2.0 ** -28, 2.0 ** 100)])
@pytest.mark.parametrize("lens,tree", [([(600, 130)], None), ([(600, 40)], None), ([(20000, 40)], None), ([(600, 60)], "tree")])
def test_a_later_scale_leaves_the_sum_of_earlier_positions(w, code, small, large, lens, tree):
    """The scales of the last positions are up to 2^160 times those before, their codes zeros: scales of values have no part in
    the log-sum, and the outputs are the earlier values times their shares.  The early values' weights are rounded by 2^-11 of
    themselves, later ones times codes of zero are zero, so that nothing but roundings of 2^-11 and the f32 scores stands
    between both sides, and fp16's smallest step in the output."""
    a = Draft(lens, 8, 2, 128, 16, "fp16", code, tree, seed=21)
    L = int(a.L[0])
    vb = a.vc.view(torch.uint8)
    for j in range(L):
        at = int(a.table[0, j // 16]), slice(None), j % 16
        a.vs[at] = small if j < 512 else large
        vb[at] = (100 if code == "int8" else 0x7e) if j < 512 else 0
    out, lse = a.run(w)
    ref, rl, spread, _ = a.reference()
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4 + 1e-6 * np.abs(rl))
    assert np.all(np.abs(f64(out) - ref) <= (2.0 ** -11 + 2e-4) * spread + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25)


def test_the_sum_of_a_long_context_of_zero_scales_stays_finite(w):
    """160 requests over the same 2^20 positions, every value's scale 0: the first 128 scores are 5.4 below the others, which is
    less than what moves a row's base.  (A tile's sum is added to the row's with one rounding of 2^-24.)"""
    L, n, d, page = 1 << 20, 17, 64, 256
    kc = torch.ones(L // page, 1, page, d, dtype=torch.int8, device="cuda")
    kc[0, :, :128] = -1
    ks = torch.full((L // page, 1, page), 2.7 * 8 / 64, device="cuda")   # scores of 2.7 and -2.7
    q = torch.ones(160 * n, 1, d, dtype=torch.float16, device="cuda")
    table = torch.arange(L // page, dtype=torch.int32, device="cuda").repeat(160, 1)
    lse = torch.zeros(160 * n, 1, device="cuda")
    out = w.w4a16_paged_attention(q, kc, torch.ones_like(kc), table, i32(np.arange(161) * n), i32([L] * 160), n, block=True,
                                  lse=lse, k_scale=ks, v_scale=torch.zeros_like(ks))
    want = 2.7 + math.log(L - 128 + 128 * math.exp(-5.4))
    assert (out == 0).all() and (lse - want).abs().max() <= 1e-4 + 1e-6 * want + L / 128 * 2.0 ** -24


# Slots that no token sees, and scales that are no numbers, in fp16: the rows' base must not take them up.
@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("fill", [3e38, float("nan"), float("-inf")])
@pytest.mark.parametrize("lens,window,tree", [([(40, 150), (3, 60)], 0, None), ([(500, 130)], 64, None), ([(700, 30)], 0, None),
                                              ([(90, 70)], 20, "tree"), ([(500, 70)], 300, "tree"), ([(99, 1), (300, 4)], 40, None)])
def test_scales_of_unseen_slots_have_no_part(w, fill, lens, window, tree, code):
    """Rows of 256 positions and more have weights of one part: bound as in test_fp16_weights_of_long_rows, with the largest
    scale that any row may see."""
    a = Draft(lens, 8, 2, 128, 16, "fp16", code, tree, seed=22)
    used = torch.zeros(a.ks.shape[0], 16, dtype=torch.bool)
    for b, L in enumerate(a.L):
        for j in range(int(L)):
            used[a.table[b, j // 16], j % 16] = True
    free = ~used[:, None].expand(-1, 2, -1).cuda()
    most = float(a.vs[~free].max()) * (127 if code == "int8" else 480)
    for c, s in ((a.kc, a.ks), (a.vc, a.vs)):
        c.view(torch.uint8)[free] = 0xff
        s[free] = fill
    out, lse = a.run(w, window)
    a.vs[free] = a.ks[free] = 0   # (the oracle does not look at them)
    ref, rl, spread, _ = a.reference(window)
    bound = (2.0 ** -11 + 2e-4) * spread + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + a.L.max() * 2.0 ** -30 * most
    assert np.all(np.abs(f64(out) - ref) <= bound)
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4 + 1e-6 * np.abs(rl))


@pytest.mark.parametrize("code", ["int8", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("lens,pos,window,tree", [([(30, 150)], 100, 0, None), ([(300, 140)], 290, 64, None), ([(700, 40)], 600, 0, None),
                                                  ([(200, 300)], 255, 0, None), ([(100, 60)], 120, 0, "tree"), ([(300, 60)], 320, 0, "tree"),
                                                  ([(300, 60)], 20, 0, "tree")])
def test_a_bad_scale_of_a_value_leaves_other_rows_alone(w, bad, lens, pos, window, tree, code):
    a = Draft(lens, 8, 2, 128, 16, "fp16", code, tree, seed=23)
    most = float(a.vs.max()) * (127 if code == "int8" else 480)
    a.vs[int(a.table[0, pos // 16]), 1, pos % 16] = bad
    out, lse = a.run(w, window)
    ref, rl, spread, _ = a.reference(window)
    got, hit = f64(out), np.isnan(ref)
    assert hit.any() and np.array_equal(np.isnan(got), hit)
    bound = (2.0 ** -11 + 2e-4) * spread + 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + a.L.max() * 2.0 ** -30 * most
    assert np.all((np.abs(got - ref) <= bound)[~hit])
    assert np.all(np.abs(f64(lse) - rl) <= 1e-4 + 1e-6 * np.abs(rl))
