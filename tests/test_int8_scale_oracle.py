"""The reference's int8 scale against exact fractions."""

from fractions import Fraction

import numpy as np

from oracle import int8_oracle as Q


def test_scales_are_the_nearest_fp32_numbers_to_the_quotient():
    rng = np.random.default_rng(41)
    top = np.concatenate([1 + np.arange(128) / 128, np.exp(rng.uniform(-60, 60, 400))]).astype(np.float32)
    _, scale = Q.quantize_rows(top[:, None])
    for t, s in zip(top, scale):
        want = Fraction(float(t)) / 127
        step = max(abs(Fraction(float(np.nextafter(s, np.float32(to)))) - Fraction(float(s))) for to in (0, np.inf))
        assert abs(Fraction(float(s)) - want) <= step / 2


def test_half_of_the_largest_value_is_63_and_a_half_steps():
    """Under a scale rounded up half of the maximum lies below the border, under one rounded down above it."""
    for sig in range(128):
        top = 1 + sig / 128
        q, s = Q.quantize_rows([[top, top / 2]])
        exact = Fraction(top) / 2 / Fraction(float(s[0]))
        assert q[0, 1] == (64 if exact >= Fraction(127, 2) else 63), sig
