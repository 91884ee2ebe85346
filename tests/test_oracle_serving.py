"""The serving operators' oracle against hand-worked values and invariants."""

import math

import numpy as np

from oracle import serving as S


def test_plan_takes_gives_back_and_drops():
    # pages of 4 tokens; stack top is 9
    table = [[3, 5, -1, -1], [1, 6, 2, -1], [-1, -1, -1, -1]]
    p = S.cache_plan(4, table, [7, 8, 9], 3, [8, 10, 0], [8, 3, 0], [1, 1, 6], 12, 64)
    # request 1 keeps 3 + 1 tokens: one page, gives back 6 and 2; request 0 takes 2 (the last
    # given back), request 2 takes 6 and then 9
    assert p["status"] == 0
    assert p["table"][0][:3] == [3, 5, 2] and p["table"][1][:1] == [1] and p["table"][2][:2] == [6, 9]
    assert p["stack"] == [7, 8]
    assert p["cu"] == [0, 1, 2, 8] and p["kv_len"] == [9, 4, 6]
    assert p["pos"] == [8, 3, 0, 1, 2, 3, 4, 5]
    assert p["slot"] == [8, 7, 24, 25, 26, 27, 36, 37]


def test_plan_refuses_whole():
    table = [[0, -1]]
    assert S.cache_plan(4, table, [], 0, [4], [4], [1], 4, 8) == {"status": 1}
    assert S.cache_plan(4, table, [1], 1, [4], [4], [5], 4, 8) == {"status": -1}  # longer than a table row
    assert S.cache_plan(4, table, [1], 1, [4], [5], [1], 4, 8) == {"status": -1}  # keeps more than it held
    assert S.cache_plan(4, table, [1], 1, [4], [4], [4], 4, 3) == {"status": -1}  # more tokens than slots


def test_rotate_quarter_turn_and_relative_positions():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    quarter = np.array([[0.0, 0.0, 1.0, 1.0]])  # cos 0, sin 1
    assert np.allclose(S.rotate(x, [0], quarter, 4), [[[-3, -4, 1, 2, 5, 6]]])
    ang = np.arange(40)[:, None] * np.array([[1.0, 0.3]])
    rope = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    g = np.random.default_rng(0)
    a, b = g.standard_normal((1, 1, 4)), g.standard_normal((1, 1, 4))
    d = [float(np.sum(S.rotate(a, [i], rope, 4) * S.rotate(b, [i + 7], rope, 4))) for i in (0, 11, 30)]
    assert max(d) - min(d) < 1e-12  # products depend on the distance alone
    assert np.array_equal(S.rotate(a, [99], rope, 4), S.rotate(a, [39], rope, 4))


def test_attend_known_weights():
    # scores 0, ln 2, ln 5: weights 1/8, 2/8, 5/8
    k = np.array([[[0.0]], [[math.log(2)]], [[math.log(5)]]])
    v = np.array([[[8.0]], [[16.0]], [[-8.0]]])
    q = np.ones((2, 1, 1))
    lo, hi = S.seen(3, 2, 0)
    assert lo.tolist() == [0, 0] and hi.tolist() == [2, 3]
    out, spread, _ = S.attend(q, k, v, lo, hi, 1.0)
    assert np.allclose(out[:, 0, 0], [8 / 3 + 32 / 3, 1 + 4 - 5]) and np.allclose(spread[1, 0, 0], 10)
    lo, hi = S.seen(3, 2, 1)
    assert np.allclose(S.attend(q, k, v, lo, hi, 1.0)[0][:, 0, 0], [16, -8])
    lo, hi = S.seen(1, 2, 0)  # a sequence shorter than its new tokens: the first sees nothing
    assert np.allclose(S.attend(q, k, v, lo, hi, 1.0)[0][:, 0, 0], [0, 8])


def test_norm_closed_forms():
    h, x = S.residual_norm([[3.0, -3.0]], [[4.0, 0.0]], w_pre=[1.0, 2.0], w_post=[1.0, 1.0], gate=[2.0, 5.0], scale=0.5, eps=0.0)
    # y / rms = [sqrt 2, 0]; h = [3 + sqrt 2, -3]
    assert np.allclose(h, [[3 + math.sqrt(2), -3]])
    r = math.sqrt(((3 + math.sqrt(2)) ** 2 + 9) / 2)
    assert np.allclose(x, [[(3 + math.sqrt(2)) / r, -6 / r]])
    assert S.residual_norm([[1.0, 1.0]], None)[1] is None
