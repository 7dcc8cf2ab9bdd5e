"""Frequencies for long contexts against what the header says of them: how often a pair turns in the first context decides
whether it is kept, stretched or between both.  Computed on the host, no GPU."""
import math

import numpy as np
import pytest

import int4_weight_only_gemm_gb300 as w
from oracle import drafts


def both(r, base, scaling, factor, length, low, high):
    got, mag = w.w4a16_rope_frequencies(r, base, scaling, factor, length, low, high, device="cpu")
    want, m = drafts.frequencies(r, base, scaling, factor, length, low, high)
    assert np.allclose(got.numpy(), want, rtol=1e-14, atol=0) and abs(mag - m) <= 2.0 ** -23 * abs(m)
    return got.numpy()


# (rotary width, base, factor, length, low, high); in the first five the last pair turns more than `low` times
RAMPS = [(128, 10000.0, 8.0, 131072.0, 1.0, 32.0), (128, 10000.0, 4.0, 65536.0, 1.0, 32.0), (64, 10000.0, 8.0, 1e6, 1.0, 32.0),
         (4, 10000.0, 8.0, 4096.0, 1.0, 32.0), (128, 500.0, 16.0, 32768.0, 1.0, 4.0), (128, 10000.0, 8.0, 4096.0, 1.0, 32.0),
         (128, 1e6, 40.0, 8192.0, 1.0, 4.0), (64, 10000.0, 4.0, 100.0, 1.0, 32.0), (64, 10000.0, 4.0, 3.0, 1.0, 32.0),
         (2, 10000.0, 4.0, 4096.0, 1.0, 32.0), (2, 10000.0, 4.0, 3.0, 1.0, 32.0), (128, 10000.0, 2.0, 1e9, 1.0, 32.0)]


@pytest.mark.parametrize("r,base,factor,length,low,high", RAMPS)
@pytest.mark.parametrize("scaling", ["ramp", "wavelength"])
def test_pairs_are_kept_or_stretched_by_their_turns(scaling, r, base, factor, length, low, high):
    plain = base ** (-2.0 * np.arange(r // 2) / r)
    turns = length * plain / (2 * math.pi)
    f = both(r, base, scaling, factor, length, low, high)
    many, few = turns > high, turns < low
    assert np.allclose(f[many], plain[many], rtol=1e-14) and np.allclose(f[few], plain[few] / factor, rtol=1e-14)
    share = (f / plain - 1) / (1 / factor - 1)   # stretched by how much: 0 .. 1
    assert np.all(share >= -1e-12) and np.all(share <= 1 + 1e-12) and np.all(np.diff(share) >= -1e-12)
    between = share[~many & ~few]
    if scaling == "wavelength":
        assert np.allclose(between, (high - turns[~many & ~few]) / (high - low), atol=1e-12)
    elif len(between) > 2:
        # linear in i, and over as many pairs as lie between `high` and `low` turns, which the base and the ends say alone,
        # with up to one more at each end: whole pairs are the line's ends.  (Not where the line begins before pair 0.)
        assert np.allclose(np.diff(between, 2), 0, atol=1e-12)
        span = r * math.log(high / low) / (2 * math.log(base))
        if many.any() and turns[-1] * base * base > low:
            assert 1 / (span + 2) - 1e-12 <= between[1] - between[0] <= 1 / span + 1e-12


@pytest.mark.parametrize("base", [1.0, 0.5, 1e-4])
def test_a_ramp_needs_pairs_that_turn_less_one_after_the_other(base):
    """At a base of 1 or below pairs turn ever more, or all alike: no pair lies between `high` and `low` turns."""
    with pytest.raises(w.W4A16Error) as e:
        w.w4a16_rope_frequencies(64, base, "ramp", 8.0, 4096.0, device="cpu")
    assert e.value.status == w.W4A16_EINVAL
    f = both(64, base, "wavelength", 8.0, 4096.0, 1.0, 32.0)   # by a pair's own turns
    plain = base ** (-2.0 * np.arange(32) / 64)
    assert np.all(f <= plain * (1 + 1e-12)) and np.all(f >= plain / 8 * (1 - 1e-12))


def test_a_line_that_ends_behind_the_last_pair():
    """128 columns, base 10000, 131072 positions: the last pair turns 2.4 times, pair 69 (there is none) once."""
    f = both(128, 10000.0, "ramp", 8.0, 131072.0, 1.0, 32.0)
    plain = 10000.0 ** (-2.0 * np.arange(64) / 128)
    first = math.floor(64 * math.log(131072 / (32 * 2 * math.pi)) / math.log(10000))
    last = math.ceil(64 * math.log(131072 / (2 * math.pi)) / math.log(10000))
    assert (first, last) == (45, 70)
    share = np.clip((np.arange(64) - first) / (last - first), 0, 1)
    assert np.allclose(f, plain * (1 - share) + plain / 8 * share, rtol=1e-13)
