"""The paged attention gives the same bits whatever ran before it: groups of query heads that do not fill a row tile, whose
last rows hold what shared memory held."""
import pytest
import torch

from test_drafts import Draft

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import int4_weight_only_gemm_gb300 as w
    return w


@pytest.mark.parametrize("code", [None, "int8", "e4m3"])
@pytest.mark.parametrize("tree", [None, "tree"])
@pytest.mark.parametrize("heads,d,dtype,window", [(28, 64, "fp16", 1024), (28, 64, "bf16", 0), (12, 128, "bf16", 0), (20, 64, "fp16", 300),
                                                  (24, 128, "fp16", 0), (44, 64, "bf16", 0)])
def test_same_bits_behind_other_calls(w, code, tree, heads, d, dtype, window):
    lens = [(1867, 50), (3337, 49), (1437, 1), (1195, 47), (2459, 33), (600, 5), (3315, 38), (130, 60)]
    a = Draft(lens, heads, 4, d, 16, dtype, code, tree, seed=41)
    junk = Draft([(400, 64)] * 24, 32, 4, d, 16, dtype, code, tree, seed=42)   # full row tiles on every SM
    first = None
    for i in range(12):
        junk.q = (torch.randn_like(junk.q, dtype=torch.float32) * 8.0 ** (i % 5)).to(junk.q.dtype)
        junk.run(w)
        out, lse = a.run(w, window)
        if first is None:
            first = out, lse
            if code is None or dtype == "bf16":   # (fp16 over 8 bits has a bound of its own for long rows)
                a.check(out, lse, window)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
