"""Attention over an 8-bit cache in fp16 with more than 16 query rows a key head: its weights are taken against a base that
the values' scales are part of, and neither the softmax's sum nor the outputs may depend on how these scales run."""
import numpy as np
import pytest
import torch

from test_drafts import Draft
from test_serving import f64

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
