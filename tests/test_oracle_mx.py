"""Pins of the microscaled 4-bit and expert oracle: values worked out by hand
and in exact rational arithmetic, and planted mistakes that the pins catch."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import mx

LEVELS = [Fraction(v) for v in ("0", "1/2", "1", "3/2", "2", "3", "4", "6")]


def _block(*head):
    x = np.zeros((1, 32))
    x[0, :len(head)] = head
    return x


def _codes(c):
    return np.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1)


def test_hand_worked_block():
    # top = 7: floor(log2 7) - 2 = 0, so the scale is 1 (byte 127) and 7 saturates at 6
    c, s = mx.quantize(_block(7.0, -0.25, 0.25001, 0.75, -1.25, 1.75, 2.5, 3.5, -5.0, 5.1, -0.0))
    assert s.tolist() == [[127]]
    # ties: .25 -> 0, .75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert _codes(c)[0, :11].tolist() == [7, 8, 1, 2, 10, 4, 4, 6, 14, 7, 8]
    # the ceil rule doubles the scale: 7 / 2 = 3.5 ties to 4
    c, s = mx.quantize(_block(7.0), "ceil")
    assert s.tolist() == [[128]] and _codes(c)[0, 0] == 6
    # 6 fits the smaller scale under either rule
    assert mx.quantize(_block(6.0), "ceil")[1].tolist() == [[127]]


@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_nearest_level_in_exact_arithmetic(rule):
    rng = np.random.default_rng(11)
    x = (rng.standard_normal((8, 64)) * 2.0 ** rng.integers(-30, 30, (8, 64))).astype(np.float32).astype(float)
    c, s = mx.quantize(x, rule)
    n, v = _codes(c), mx.dequantize(c, s)
    for r in range(8):
        for k in range(64):
            b = int(s[r, k // 32]) - 127
            top = max(abs(Fraction(t)) for t in x[r, k // 32 * 32:][:32])
            scale = Fraction(2) ** b
            if rule == "floor":
                assert 4 * scale <= top < 8 * scale
            else:
                assert 3 * scale < top <= 6 * scale
            a = abs(Fraction(x[r, k])) / scale
            d = [abs(a - q) for q in LEVELS]
            i = int(n[r, k]) & 7
            assert d[i] == min(d) and (d.count(min(d)) == 1 or i % 2 == 0)
            assert Fraction(v[r, k]) == (-1 if n[r, k] & 8 else 1) * LEVELS[i] * scale


def test_zero_inf_and_nan_blocks():
    x = np.zeros((1, 96))
    x[0, 40], x[0, 70] = np.inf, np.nan
    c, s = mx.quantize(x)
    assert s.tolist() == [[0, 255, 255]] and not c.any()
    v = mx.dequantize(c, s)
    assert (v[0, :32] == 0).all() and np.isnan(v[0, 32:]).all()


def test_low_nibble_is_the_even_value():
    c, _ = mx.quantize(_block(1.0, 4.0))
    assert c[0, 0] == 0x62


def test_route_by_hand():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0], [3.0, 1.0, 3.0, 1.0]]))
    ids, w = mx.route(l, 2)
    assert ids.tolist() == [[1, 2], [0, 2]]                     # equal ones: the lower first
    assert np.allclose(w, [[2 / 3, 1 / 3], [0.5, 0.5]])
    ids, w = mx.route(l, 2, renorm=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5], [0.75, 0.75]])
    # a bias moves the choice, not the weight
    ids, w = mx.route(l, 1, bias=[1.0, 0, 0, 0], renorm=False)
    assert ids.tolist() == [[0], [0]] and np.allclose(w, [[1 / 8], [3 / 8]])
    # groups {0, 1}, {2, 3}: sums of the two best 5 / 8 and 3 / 8, then 4 / 8 and 4 / 8
    ids, _ = mx.route(l, 2, groups=2, top_groups=1, group_best=2)
    assert ids.tolist() == [[1, 0], [0, 1]]


def test_route_sigmoid_and_masked_rows():
    l = np.array([[0.0, np.log(3.0), -np.inf], [-np.inf] * 3, [np.nan, 0.0, 0.0]])
    ids, w = mx.route(l, 3, score="sigmoid")
    assert ids.tolist() == [[1, 0, -1], [-1, -1, -1], [1, 2, -1]]
    assert np.allclose(w, [[0.6, 0.4, 0], [0, 0, 0], [0.5, 0.5, 0]])


def test_plan_by_hand():
    o, p = mx.plan([[2, 0], [-1, 2], [0, 7]], 3)
    assert o.tolist() == [0, 2, 2, 4] and p.tolist() == [1, 4, 0, 3, -1, -1]


def test_moe_mlp_in_exact_small_integers():
    # silu(0) = 0 kills a unit whatever its up value; big gates pass it through
    x = np.array([[1.0, 2.0]])
    gate_up = np.array([[[0, 0], [60, 60], [5, 5], [1, 1]]], float)   # gates 0 and 180, ups 15 and 3
    down = np.array([[[7, 1], [9, -2]]], float)
    y, err = mx.moe_mlp(x, gate_up, down, np.array([[0, -1]]), np.array([[0.5, 3.0]]), 0, 1, 1)
    assert np.allclose(y, [[0.5 * 540, -540.0]]) and (err < 1e-2).all()


def test_planted_mistakes_are_seen():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((4, 64))
    c, s = mx.quantize(x)
    v = mx.dequantize(c, s)
    assert np.abs(mx.dequantize((c >> 4) | (c << 4), s) - v).max() > 0.1      # nibbles exchanged
    assert np.abs(mx.dequantize(c, s[:, ::-1]) - v).max() > 0                 # scales reversed
    assert np.abs(mx.dequantize(c ^ 0x88, s) + v).max() == 0                  # signs flipped
