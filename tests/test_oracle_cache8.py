"""The 8-bit cache's definitions pinned by hand-worked values and invariants."""

import numpy as np
import pytest

from oracle import serving as S


def test_codes_by_hand():
    v = S.e4m3_values()
    for code, value in [(0, 0.0), (1, 2.0 ** -9), (7, 7 * 2.0 ** -9), (8, 2.0 ** -6), (0x38, 1.0), (0x3c, 1.5), (0x40, 2.0), (0x7e, 448.0), (0x77, 240.0),
                        (0xb8, -1.0), (0x81, -(2.0 ** -9)), (0xfe, -448.0)]:
        assert v[code] == value, hex(code)
    assert np.isnan(v[[0x7f, 0xff]]).all() and np.isfinite(np.delete(v, [0x7f, 0xff])).all()
    assert (np.diff(v[:127]) > 0).all()


@pytest.mark.parametrize("top,b", [(448.0, 127), (448.0001, 128), (1.75, 119), (1.76, 120), (1.0, 119), (0.0, 10), (1e-45, 10), (3.4e38, 246),
                                   (448 * 2.0 ** 119, 246), (448 * 2.0 ** 118, 245), (448 * 2.0 ** -117, 10), (449 * 2.0 ** -117, 11)])
def test_a_rows_power_of_two(top, b):
    assert S.quantise(np.array([[0.0, -top, top / 3]]))[1][0] == b


def test_rounding_ties_and_ends():
    # with a 448 in the row the power is 2^0 and values are code values
    row = [448.0, 17.0, 19.0, 17.001, 0.4 * 2.0 ** -9, 0.5 * 2.0 ** -9, 0.51 * 2.0 ** -9, 1.5 * 2.0 ** -9, -17.0, 240.0]
    codes, b = S.quantise(np.array(row))
    assert b == 127
    assert S.stand_for(codes, b).tolist() == [448.0, 16.0, 20.0, 18.0, 0.0, 0.0, 2.0 ** -9, 2 * 2.0 ** -9, -16.0, 240.0]


def test_what_is_not_finite():
    x = np.array([[np.inf, 1.0, -np.inf, np.nan], [3.4e38, 1.0, 0.0, -3.4e38]])
    codes, b = S.quantise(x)
    assert b.tolist() == [119, 246]
    got = S.stand_for(codes, b)
    assert np.isnan(got[0, [0, 2, 3]]).all() and got[0, 1] == 1.0
    assert got[1].tolist() == [448 * 2.0 ** 119, 0.0, 0.0, -448 * 2.0 ** 119]


@pytest.mark.parametrize("seed", range(5))
def test_error_of_a_value(seed):
    g = np.random.default_rng(seed)
    x = g.standard_normal((50, 128)) * np.exp(3 * g.standard_normal((50, 1)))
    codes, b = S.quantise(x)
    b2 = 2.0 ** (b.astype(float) - 127)[:, None]
    top = np.abs(x).max(1, keepdims=True)
    assert (top <= 448 * b2).all() and (top > 224 * b2).all()
    # half a step: 2^-4 of the value, or half of the smallest code where that is more
    assert (np.abs(S.stand_for(codes, b) - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * b2)).all()
    again = S.quantise(S.stand_for(codes, b))
    assert np.array_equal(S.stand_for(*again), S.stand_for(codes, b))
