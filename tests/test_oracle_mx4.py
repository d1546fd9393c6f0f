"""Pins of the microscaled 4-bit oracle that need nothing but arithmetic:
hand-worked blocks, every code, ties, the scale rule at its borders, exact
rational sums, the router's order."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4 as X


def block(values):
    return np.array(values + [0.0] * (32 - len(values)), np.float32)[None]


def test_hand_worked_block():
    # amax 7: floor(log2 7) - 2 = 0, scale 1 (byte 127); 7 saturates at 6
    c, s = X.quantize(block([7.0, -1.25, 0.25, 0.26, 2.5, -3.5, 5.0, 5.1, -0.0]))
    assert s.tolist() == [[127]]
    assert c[0, :9].tolist() == [7, 8 | 2, 0, 1, 4, 8 | 6, 6, 7, 8]
    p, q = X.planes(c, s)
    assert p[0, :5].tolist() == [0xA7, 0x10, 0xE4, 0x76, 0x08] and q.tolist() == [[127]]
    assert X.dequantize(c, s)[0, :4].tolist() == [6.0, -1.0, 0.0, 0.5]


def test_every_code_returns_itself():
    for s in (0, 1, 100, 127, 200, 252):
        v = np.concatenate([X.MAGNITUDES, -X.MAGNITUDES, X.MAGNITUDES, -X.MAGNITUDES])[None] * 2.0 ** (s - 127)
        c, t = X.quantize(v.astype(np.float64))
        assert t.tolist() == [[s]]
        assert (c[0, :16] == np.arange(16)).all()


def test_ties_go_to_the_even_mantissa():
    ties = [(0.25, 0), (0.75, 2), (1.25, 2), (1.75, 4), (2.5, 4), (3.5, 6), (5.0, 6)]
    assert X.nearest_code(np.array([t for t, _ in ties])).tolist() == [c for _, c in ties]
    eps = 2.0 ** -40
    assert X.nearest_code(np.array([t - eps for t, _ in ties])).tolist() == list(range(7))
    assert X.nearest_code(np.array([t + eps for t, _ in ties])).tolist() == list(range(1, 8))


@pytest.mark.parametrize("amax,byte", [(4.0, 127), (7.999, 127), (8.0, 128), (3.999, 126), (0.0, 0), (2.0 ** -125, 0),
                                       (2.0 ** -124, 1), (2.0 ** -149, 0), (3.0e38, 252)])
def test_scale_byte(amax, byte):
    assert X.quantize(block([amax]))[1].tolist() == [[byte]]


def test_non_finite_blocks():
    for bad in (np.inf, -np.inf, np.nan):
        x = np.concatenate([block([1.0, bad]), block([1.0])], 1)
        c, s = X.quantize(x)
        assert s[0, 0] == 255 and not c[0, :32].any() and s[0, 1] == 125
        assert np.isnan(X.dequantize(c, s)[0, :32]).all() and X.dequantize(c, s)[0, 32] == 1.0


def test_error_is_at_most_half_a_step():
    x = np.random.default_rng(3).standard_normal((64, 96)).astype(np.float32)
    c, s = X.quantize(x)
    v = X.dequantize(c, s)
    unit = np.repeat(np.exp2(s.astype(float) - 127), 32, 1)
    a = np.abs(x) / unit
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, np.where(a <= 6, 1.0, np.maximum(a - 6, 1.0)))) * unit
    assert (np.abs(v - x) <= half).all()


def test_bf16_bits_widen():
    assert X.widen(np.array([0x3F80, 0xC000, 0x7F80], np.uint16)).tolist() == [1.0, -2.0, np.inf]


def test_product_against_rational_sums():
    rng = np.random.default_rng(5)
    c, s = rng.integers(0, 16, (3, 64)).astype(np.uint8), rng.integers(120, 135, (3, 2)).astype(np.uint8)
    x = rng.standard_normal((2, 64)).astype(np.float16).astype(np.float64)
    w = X.dequantize(c, s)
    y, a = X.product(w, x)
    for m in range(2):
        for n in range(3):
            t = [Fraction(float(w[n, k])) * Fraction(float(x[m, k])) for k in range(64)]
            assert abs(float(sum(t)) - y[m, n]) <= 64 * 2.0 ** -52 * a[m, n]
            assert abs(float(sum(abs(v) for v in t)) - a[m, n]) <= 64 * 2.0 ** -52 * a[m, n]


def test_route_order_and_weights():
    W = np.array([[1.0], [3.0], [3.0], [-2.0], [np.nan]])
    ids, p, _ = X.route(np.array([[1.0]]), W, 3, True)
    assert ids.tolist() == [[1, 2, 0]]
    e = np.exp([0.0, 0.0, -2.0])
    assert np.allclose(p[0], e / e.sum(), rtol=1e-15)
    assert np.isnan(X.route(np.array([[1.0]]), W, 3, False)[1]).all()
    ids, p, _ = X.route(np.array([[1.0]]), W[:4], 4, False)
    assert ids.tolist() == [[1, 2, 0, 3]] and abs(p.sum() - 1) < 1e-15


def test_layer_of_one_expert_is_its_ffn():
    rng = np.random.default_rng(7)
    x, g, u, d = (rng.standard_normal(s) for s in ((2, 32), (1, 64, 32), (1, 64, 32), (1, 32, 64)))
    y, bound = X.moe_layer(x, g, u, d, np.zeros((2, 1), np.int32), np.ones((2, 1)))
    z = x @ g[0].T
    assert np.allclose(y, (z / (1 + np.exp(-z)) * (x @ u[0].T)) @ d[0].T, rtol=1e-12)
    assert (bound > 0).all() and (bound < 1e-2 * np.abs(y).max()).all()


def test_values_past_fp32():
    """Code times scale up to 6 * 2^127; infinite only as fp32 or bf16 hold it."""
    c, s = np.full((4, 32), 7, np.uint8), np.array([[252], [253], [254], [255]], np.uint8)
    c[:, 1], c[:, 2] = 8 | 4, 2
    v = X.values(c, s)
    assert v[:3, :3].tolist() == [[6 * 2.0 ** (b - 127), -(2.0 ** (b - 126)), 2.0 ** (b - 127)] for b in (252, 253, 254)]
    d = X.dequantize(c, s)
    assert d[:3, :3].tolist() == [v[0, :3].tolist(), [np.inf, -(2.0 ** 127), 2.0 ** 126], [np.inf, -np.inf, 2.0 ** 127]]
    assert np.isnan(v[3]).all() and np.isnan(d[3]).all()
