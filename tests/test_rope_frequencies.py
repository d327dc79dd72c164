"""Frequencies by parts, pair by pair (no GPU)."""
import math

import numpy as np
import pytest

import compressed_attention_adaptive_gb300 as mita
from compressed_attention_adaptive_gb300 import build as mita_build


@pytest.fixture(scope="module", autouse=True)
def lib():
    mita_build.build()
    return mita.lib()


@pytest.mark.parametrize("original,low,high,factor,want", [
    (8192.0, 1.0, 4.0, 8.0, 1.0),                       # pair 0 turns 1304 times: as it is
    (20.0 * math.pi, 1.0, 4.0, 8.0, 1.0),               # ten times
    (5.0 * math.pi, 1.0, 4.0, 8.0, 0.5 + 0.5 / 8.0),    # 2.5 times, the middle of the ramp
    (math.pi, 1.0, 4.0, 8.0, 1.0 / 8.0),                # half a turn: slowed altogether
])
def test_first_pair_by_parts(original, low, high, factor, want):
    """A handful of roundings of 2^-53 on a number of at most 1, times the ramp's slope of 1/3."""
    got = mita.mita_rope_frequencies(64, scaling=mita.ROPE_PARTS, factor=factor, original=original, low=low, high=high)
    assert abs(got[0] - want) <= 16 * 2.0 ** -53
    plain = np.array(mita.mita_rope_frequencies(64))
    turns = original * plain / (2 * math.pi)
    f = np.array(got)
    fast, slow = turns >= high * (1 + 1e-12), turns <= low * (1 - 1e-12)
    assert np.array_equal(f[fast], plain[fast])
    assert np.all(np.abs(f[slow] - plain[slow] / factor) <= plain[slow] * 4 * 2.0 ** -53)
    between = ~(fast | slow)
    assert np.all((f[between] <= plain[between]) & (f[between] >= plain[between] / factor * (1 - 4 * 2.0 ** -53)))
