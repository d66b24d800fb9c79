"""The stretched frequencies of ROPE_YARN against values worked out by hand: between pairs `low` and
`high` the share r of f_i that is divided by the factor rises from 0 to 1.  The pair that makes t turns over
L positions is rope_dim / 2 * ln(L / (2 pi t)) / ln(theta); low is that of the fast turns rounded down,
high that of the slow ones rounded up, within [0, rope_dim - 1].
"""
from fractions import Fraction

import pytest

import kv_norm_rope_gb300 as k

CASES = [
    # rope_dim, theta, factor, positions, fast and slow turns, low, high
    (64, 1e4, 16.0, 65536.0, 32.0, 1.0, 20, 33),    # 20.11, 32.15: no pair is stretched whole
    (64, 1e4, 32.0, 131072.0, 32.0, 1.0, 22, 35),   # 22.51, 34.55
    (64, 1e4, 4.0, 262144.0, 32.0, 1.0, 24, 37),    # 24.92, 36.96
    (128, 1e4, 16.0, 65536.0, 32.0, 1.0, 40, 65),   # 40.21, 64.29
    (64, 1e4, 40.0, 4096.0, 32.0, 1.0, 10, 23),     # 10.47, 22.51: the last nine are
    (64, 1.6e5, 16.0, 65536.0, 32.0, 1.0, 15, 25),  # 15.45, 24.71
    (64, 1e4, 8.0, 100.0, 32.0, 1.0, 0, 10),        # below 0, 9.61
    (8, 100.0, 8.0, 1e5, 1000.0, 1.0, 2, 7),        # 2.40, 8.40: past rope_dim - 1
    (8, 100.0, 8.0, 1e8, 32.0, 1.0, 11, 12),        # 11.39, 14.40: every pair is fast
]


@pytest.mark.parametrize("dim,theta,factor,positions,fast,slow,low,high", CASES)
def test_ramp(dim, theta, factor, positions, fast, slow, low, high):
    plain = k.rope_frequencies(dim, theta)
    got = k.rope_frequencies(dim, theta, k.ROPE_YARN, factor, positions, fast, slow)
    for i, (f, g) in enumerate(zip(plain, got)):
        r = min(max(Fraction(i - low, high - low), 0), 1)
        # two roundings of f's parts and their sum's, 2^-53 each
        want = float(1 - r + r / Fraction(factor)) * f
        assert abs(g - want) <= 2.0 ** -50 * want, (i, g / f, r)


def test_the_last_pair_of_a_long_original_context():
    plain, yarn = k.rope_frequencies(64), k.rope_frequencies(64, 10000.0, k.ROPE_YARN, 16.0, 65536.0)
    assert abs(yarn[31] / plain[31] - (2 / 13 + 11 / 13 / 16)) <= 2.0 ** -50
    assert yarn[20] == plain[20] and yarn[21] < plain[21]
