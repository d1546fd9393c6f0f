"""The oracle of rotary positions, the paged cache and attention, pinned by values worked by hand."""
import math

import numpy as np
import pytest

from oracle import attn as A
from oracle import formats as F


def test_quarter_turns():
    """A pair turned by pi / 2, pi and 3 pi / 2; the rest of the head copied."""
    x = np.array([[[3.0, 5.0, 7.0, 11.0, 13.0, 17.0]]])
    f = np.array([np.pi / 2, np.pi])
    assert np.allclose(A.rope(x, [1], f, 2.0, True), [[[-10, 6, -14, -22, 13, 17]]], atol=1e-14)
    assert np.allclose(A.rope(x, [1], f, 2.0, False), [[[-14, -10, 6, -22, 13, 17]]], atol=1e-14)
    assert np.allclose(A.rope(x, [3], f, 1.0, True), [[[5, -3, -7, -11, 13, 17]]], atol=1e-14)
    assert np.allclose(A.rope(x, [-1], f, 1.0, True), [[[5, -3, -7, -11, 13, 17]]], atol=1e-14)
    assert np.array_equal(A.rope(x, [0], f, 1.0, False), x)


def test_rotation_depends_on_distance_alone():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((2, 1, 1, 64))
    f, m = A.freqs("none", 64, 1e4)
    dots = [float((A.rope(q, [p + 37], f, m, False) * A.rope(k, [p], f, m, False)).sum()) for p in (0, 5, 1000)]
    assert np.allclose(dots, dots[0], rtol=1e-11)


def test_frequencies():
    f, m = A.freqs("none", 4, 100.0)
    assert np.allclose(f, [1, 0.1]) and m == 1
    assert np.allclose(A.freqs("linear", 4, 100.0, 8.0)[0], [1 / 8, 0.1 / 8])
    assert np.allclose(A.freqs("ntk", 4, 100.0, 4.0)[0], [1, 1 / 40])
    # 2 pi * 16.5 positions: 16.5 turns of the first pair, halfway between 1 and 32; 1.65 of the second
    f, m = A.freqs("yarn", 4, 100.0, 10.0, 2 * np.pi * 16.5)
    g = 0.65 / 31
    assert np.allclose(f, [0.5 + 0.05, g * 0.1 + (1 - g) * 0.01]) and math.isclose(m, 1 + 0.1 * math.log(10))


def test_places_by_hand():
    assert A.place("f16", False, 0, 0) == 0 and A.place("f16", True, 0, 0) == 0
    # position 13: r = 4 * 1 + 1 = 5, t = 1; channel 41: block 1, piece 1, element 1
    assert A.place("f16", False, 13, 41) == (1 * 2 + 1) * 512 + (1 * 16 + 5) * 8 + 1
    assert A.place("q8_0", False, 13, 41) == 1024 + (1 * 16 + 5) * 16 + 8 + 1
    # V: channel 41 = 2 * 16 + 9; position 13 = 8 + 5
    assert A.place("bf16", True, 13, 41) == 2 * 512 + (1 * 16 + 9) * 8 + 5
    assert A.place("q8_0", True, 13, 41) == 1024 + (1 * 16 + 9) * 16 + 0 + 5
    assert A.place("q8_0", True, 13, 63) == 1024 + (1 * 16 + 15) * 16 + 8 + 5


@pytest.mark.parametrize("kind", ["f16", "bf16", "q8_0"])
@pytest.mark.parametrize("is_v", [False, True])
def test_put_and_get(kind, is_v):
    rng = np.random.default_rng(2)
    region = np.full(A.region_bytes(kind, 64), 0x55, np.uint8)
    rows = rng.standard_normal((32, 64))
    for p in range(32):
        A.put(region, kind, is_v, p, rows[p])
    got = A.get(region, kind, is_v)
    if kind == "q8_0":
        f = F.quantize("q8_0", rows.astype(np.float32))
        assert np.array_equal(got, F.dequantize("q8_0", f))
    else:
        assert np.array_equal(got, A.widen(A.narrow(rows, kind)))


def test_bf16_rounding():
    x = np.array([1.0, 1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1 + 2.0 ** -8 + 2.0 ** -20, -2.5, np.inf, np.nan, 3.4e38])
    got = A.widen(A.bf16_bits(x))
    assert np.array_equal(got, [1, 1, 1 + 2.0 ** -6, 1 + 2.0 ** -7, -2.5, np.inf, np.nan, np.inf], equal_nan=True)


def test_blocks_without_a_finite_scale():
    x = np.ones((4, 64), np.float32)
    x[0, 3], x[1, 40], x[2, 0] = np.inf, np.nan, 1e7
    q, d = A.q8_blocks(x)
    assert np.isnan(d).tolist() == [[True, False], [False, True], [True, False], [False, False]]
    assert (q[np.repeat(np.isnan(d), 32, -1)] == 0).all() and (q[3] == 127).all()


def test_visibility():
    assert A.visible(2, 5, 0).tolist() == [True, True, True, False, False]
    assert A.visible(3, 5, 2).tolist() == [False, False, True, True, False]
    assert not A.visible(-1, 4, 0).any()
    # three new tokens from position 4 on; the last sees the first and itself
    assert A.visible(6, 7, 0, 0b101, 4).tolist() == [True] * 5 + [False, True]
    assert A.visible(6, 7, 3, 0b001, 4).tolist() == [False] * 4 + [True, False, False]


def test_attention_by_hand():
    """Weights 1 : 3 by a score of ln 3; nothing seen; scores of minus infinity; a NaN."""
    k, v = np.array([[0.0, 0], [math.log(3) / 2, 0]]), np.array([[1.0, 2], [5, -6]])
    q = np.array([4.0, 1])
    out, mass, *_ = A.attend(q, k, v, 0.5, np.array([True, True]))
    assert np.allclose(out, [4, -4]) and np.allclose(mass, [4, 5])
    assert np.array_equal(A.attend(q, k, v, 0.5, np.array([False, True]))[0], [5, -6])
    assert not A.attend(q, k, v, 0.5, np.array([False, False]))[0].any()
    assert not A.attend(q, np.full((2, 2), -np.inf), v, 0.5, np.array([True, True]))[0].any()
    assert np.isnan(A.attend(q, np.array([[np.nan, 0], [0, 0]]), v, 0.5, np.array([True, True]))[0]).all()


def test_tolerance_by_hand():
    """Half a step of the output and the mass times the relative errors."""
    out, mass = np.array([2.0]), np.array([3.0])
    got = A.attention_tolerance(out, mass, 0.25, np.array([4.0]), 16, "bf16", 0.125)[0]
    rel = 0.5 + 2.0 ** -20 + 64 * 2.0 ** -24 + 0.125
    assert math.isclose(got, 2.0 ** -8 * (2 + 3 * rel) + 3 * rel + 4 * 2.0 ** -25 + 2.0 ** -25)
