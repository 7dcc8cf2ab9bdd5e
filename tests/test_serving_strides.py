"""Strides of the serving operators' arrays: what the entry points take and refuse, checked without a GPU through the
C ABI's refusals, and what they compute with the strides of dimensions of one entry."""
import numpy as np
import pytest
import torch

import int4_weight_only_gemm_gb300 as w
from test_serving_oracle import ATTN, PTR, attn_base, call, fields

WRITE = fields("k v slots kc vc kt kh vt vh kcp kch kcs vcp vch vcs T H d pages page dtype flags reserved")


def write_base():
    return dict(zip(WRITE, PTR[:5] + [256, 128, 256, 128, 4096, 2048, 128, 4096, 2048, 128, 8, 2, 128, 64, 16, 0, 1, 0]))


@pytest.fixture(scope="module", autouse=True)
def built():
    from int4_weight_only_gemm_gb300 import _build
    _build.build()


def test_attention_strides_of_zero():
    """Expanded heads, tokens or pages: refused whatever the lengths are, not by one of the two kernels only."""
    do = lambda **c: call(w, "w4a16_paged_attention", w._ATTN_ARGS, ATTN, attn_base(), **c)  # noqa: E731
    for s in ("qt", "qh", "ot", "oh", "kcp", "kch", "kcs", "vcp", "vch", "vcs"):
        for max_q in (1, 300):
            assert do(**{s: 0, "max_q": max_q}) == w.W4A16_EINVAL, s
        assert do(**{s: 4}) == w.W4A16_EALIGN, s


def test_write_strides_of_zero():
    do = lambda **c: call(w, "w4a16_kv_write", w._WRITE_ARGS, WRITE, write_base(), **c)  # noqa: E731
    for s in ("kcp", "kch", "kcs", "vcp", "vch", "vcs"):
        assert do(**{s: 0}) == w.W4A16_EINVAL, s


def test_strides_of_one_entry_are_not_looked_at():
    """The checks behind theirs answer: arrays that overlap, another stride, a missing workspace (on a GPU)."""
    do = lambda **c: call(w, "w4a16_paged_attention", w._ATTN_ARGS, ATTN, attn_base(), **c)  # noqa: E731
    one = dict(T=1, qt=3, ot=-5, pages=1, kcp=7, vcp=0)
    assert do(out=attn_base()["q"], **one) == w.W4A16_EINVAL
    assert do(qh=12, **one) == w.W4A16_EALIGN
    assert do(ws=0, **one) in (w.W4A16_EWORKSPACE, w.W4A16_ECUDA)


@pytest.mark.gpu
@pytest.mark.parametrize("past,new", [(37, 1), (37, 40)])
def test_one_head_one_page_one_token(past, new):
    """PyTorch may give a dimension of one entry any stride."""
    g = torch.Generator("cuda").manual_seed(3)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    q, k, v = rnd(new, 1, 64), rnd(past + new, 1, 64), rnd(past + new, 1, 64)
    odd = lambda t, d, s: torch.as_strided(t, t.shape, [s if i == d else x for i, x in enumerate(t.stride())])  # noqa: E731
    kc, vc = torch.zeros(2, 1, 1, 128, 64, dtype=torch.bfloat16, device="cuda")
    kc, vc = odd(odd(kc, 0, 3), 1, 0), odd(odd(vc, 0, 0), 1, 5)
    w.w4a16_kv_write(odd(k, 1, 3), odd(v, 1, 0), torch.arange(past + new, dtype=torch.int32, device="cuda"), kc, vc)
    q = odd(q, 1, 1)
    if new == 1:
        q = odd(q, 0, 9)
    out = w.w4a16_paged_attention(q, kc, vc, i32([[0]]), i32([0, new]), i32([past + new]), new)
    s = q.double()[:, 0] @ k.double()[:, 0].T / 8
    s = s.masked_fill(torch.arange(past + new, device="cuda")[None] > past + torch.arange(new, device="cuda")[:, None], -np.inf)
    p = torch.softmax(s, 1)
    want, spread = p @ v.double()[:, 0], p @ v.double()[:, 0].abs()
    assert ((out.double()[:, 0] - want).abs() <= (2.0 ** -9 + 2e-4) * spread + 2.0 ** -9 * want.abs()).all()
