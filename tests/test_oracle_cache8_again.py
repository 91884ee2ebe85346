"""Rows of the 8-bit cache that are read back and quantised again: the same values, though not always
the same codes."""

import numpy as np
import pytest

from oracle import serving as S


@pytest.mark.parametrize("top,lower", [(1.75, False), (1.7500001, True), (1.78, True), (1.8125, True), (1.8125001, False), (1.9, False), (1.0, False),
                                       (1.99, False), (1.5, False)])
@pytest.mark.parametrize("e", [-100, 0, 60])
def test_a_magnitude_that_is_rounded_down_to_the_power_before(top, lower, e):
    """1.75 times a power of two is the largest code of one byte and half of that of the next: a row whose
    largest magnitude is rounded down to it (up to 1.8125, the tie) has the lower byte the second time,
    and twice the codes' values."""
    x = np.array([top, -top / 3, top / 900, top / 50000, 0.0]) * 2.0 ** e
    codes, b = S.quantise(x)
    again, b2 = S.quantise(S.stand_for(codes, b))
    assert np.array_equal(S.stand_for(again, b2), S.stand_for(codes, b))
    assert b2 == b - lower and np.array_equal(again, codes) != lower
    third, b3 = S.quantise(S.stand_for(again, b2))
    assert b3 == b2 and np.array_equal(third, again)


@pytest.mark.parametrize("seed", range(5))
def test_values_stay_whatever_the_row(seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((400, 64)) * np.exp(20 * g.standard_normal((400, 1)))
    x[::7, 3], x[::11, 5], x[::13] = np.inf, np.nan, 0.0
    codes, b = S.quantise(x)
    once = S.stand_for(codes, b)
    again, b2 = S.quantise(once)
    assert np.array_equal(S.stand_for(again, b2), once, equal_nan=True)
    assert set((b.astype(int) - b2).tolist()) <= {0, 1} and (b != b2).any()
