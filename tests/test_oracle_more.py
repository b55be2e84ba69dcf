"""Pins of the oracle's 4-bit format and verification of drafted tokens, worked out by hand or with another method."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import drafts, mx4


def test_quantize_hand_worked():
    # amax 6 .. 7.99: scale 1; 8: scale 2
    codes, s = mx4.quantize_block([6.0, -5.0, 5.1, 0.25, 0.26, -0.75, 1.25, 1.75, 2.5, 3.5, 4.9, -0.0])
    assert s == 127
    # 5 is a tie of 4 (code 6) and 6 (code 7); 0.25 of 0 and 0.5; 0.75 of 0.5 (1) and 1 (2); 1.25 of 1 (2) and 1.5 (3);
    # 1.75 of 1.5 (3) and 2 (4); 2.5 of 2 (4) and 3 (5); 3.5 of 3 (5) and 4 (6)
    assert list(codes) == [7, 14, 7, 0, 1, 10, 2, 4, 4, 6, 6, 8]
    codes, s = mx4.quantize_block([7.999, 1.0])
    assert s == 127 and list(codes) == [7, 2]  # more than 6 stays 6
    codes, s = mx4.quantize_block([8.0, 1.0, 0.4])
    assert s == 128 and list(codes) == [6, 1, 0]
    assert mx4.quantize_block([0.0, -0.0]) [1] == 0
    codes, s = mx4.quantize_block([2.0 ** -149, 2.0 ** -127])  # the smallest scale is 2^-127
    assert s == 0 and list(codes) == [0, 2]
    for bad in (math.inf, -math.inf, math.nan):
        codes, s = mx4.quantize_block([1.0, bad])
        assert s == 255 and not codes.any()


def test_codes_are_nearest_in_exact_arithmetic():
    rng = np.random.default_rng(0)
    x = np.float32(rng.standard_normal((40, 32)) * np.exp2(rng.integers(-130, 120, (40, 1))))
    codes, scales = mx4.quantize(x)
    values = mx4.dequantize(codes, scales)
    for r in range(40):
        unit = Fraction(2) ** (int(scales[r, 0]) - 127)
        assert max(abs(Fraction(float(v))) for v in x[r]) < 8 * unit or scales[r, 0] == 0
        for v, q in zip(x[r], values[r]):
            v, q = Fraction(float(v)), Fraction(float(q))
            best = min(abs(abs(v) - Fraction(float(c)) * unit) for c in mx4.VALUES)
            assert abs(v - q) == best


def test_bytes_and_ragged_last_block():
    x = np.arange(1.0, 36.0)[None]
    codes, scales = mx4.quantize(x)
    assert codes.shape == (1, 32) and scales.shape == (1, 2)
    # 33, 34, 35 under scale 8: 4.125, 4.25, 4.375 -> 4 (code 6); the even element in the low half; zeros behind
    assert scales[0, 1] == 130 and list(codes[0, 16:19]) == [0x66, 0x06, 0x00] and not codes[0, 19:].any()
    assert mx4.dequantize(codes, scales)[0, 32:36].tolist() == [32.0, 32.0, 32.0, 0.0]


def test_matmul_is_the_sum_of_products():
    rng = np.random.default_rng(1)
    x, w = mx4.quantize(rng.standard_normal((2, 40))), mx4.quantize(rng.standard_normal((3, 40)))
    y, mag = mx4.matmul(mx4.dequantize(*x), mx4.dequantize(*w))
    a, b = mx4.dequantize(*x), mx4.dequantize(*w)
    assert y[1, 2] == pytest.approx(math.fsum(a[1] * b[2]), rel=1e-15) and (mag >= np.abs(y)).all()


def test_draw_is_the_inverse_of_the_running_sum():
    share = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    for u, want in ((0.0, 1), (0.2499, 1), (0.25, 3), (0.7499, 3), (0.75, 4), (0.9999, 4), (1.0, 4), (-1.0, 1),
                    (math.nan, 1)):
        assert drafts.draw(share, u) == want


def test_verification_keeps_the_target_distribution():
    """Over a grid of both random numbers every token comes out as often as the target says, whatever the draft says."""
    p, q = np.array([0.5, 0.25, 0.125, 0.125]), np.array([0.125, 0.5, 0.25, 0.125])
    with np.errstate(divide="ignore"):
        target, draft = np.log(np.stack([p, p]))[None], np.log(q)[None, None]
    n, got = 64, np.zeros(4)
    for x in range(4):
        for i in range(n):
            for j in range(n):
                u = np.array([[(i + 0.5) / n, (j + 0.5) / n]])
                got[drafts.verify(target, draft, np.array([[x]]), None, u)[1][0, 0]] += q[x] / n / n
    assert np.abs(got - p).max() < 0.02


def test_verification_stops_where_it_must():
    z = np.zeros((1, 3, 4))
    tokens, u = np.array([[1, 2]]), np.array([[0.1, 0.1, 0.6]])
    a, t, lp = drafts.verify(z, None, tokens, None, u)  # p = 1/4 each, the draft certain: 0.1 < 0.25 twice
    assert a[0] == 2 and t[0].tolist() == [1, 2, 2] and np.allclose(lp[0], math.log(0.25))
    a, t, lp = drafts.verify(z, None, tokens, np.array([1]), u)
    assert a[0] == 1 and t[0].tolist() == [1, 2, -1] and lp[0, 2] == 0
    a, t, _ = drafts.verify(z, None, tokens, None, np.array([[0.1, 0.3, 0.34]]))  # 2 falls: the rest is 0, 1, 3
    assert a[0] == 1 and t[0].tolist() == [1, 1, -1]
    a, t, _ = drafts.verify(z, None, np.array([[1, 4]]), None, u)
    assert a[0] == 1 and t[0].tolist() == [1, 2, -1]
    a, t, _ = drafts.verify(z, None, tokens, np.array([-1]), u)
    assert a[0] == 0 and t[0].tolist() == [-1, -1, -1]
    z[0, 1, 3] = np.nan
    a, t, lp = drafts.verify(z, None, tokens, None, u)
    assert a[0] == 1 and t[0].tolist() == [1, -1, -1] and np.isnan(lp[0, 1]) and lp[0, 2] == 0
    a, t, _ = drafts.verify(z, None, tokens, None, np.array([[0.5, 0.1, 0.6]]))  # the NaN row is not needed
    assert a[0] == 0 and t[0].tolist() == [2, -1, -1]
