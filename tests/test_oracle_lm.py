"""The 64-bit oracle of the language-model operators against central
differences and closed forms (no GPU)."""
import math

import numpy as np
import pytest

from oracle import lm

H = 1e-5
# a central difference in 64 bits: truncation H^2 f''' / 6 (f''' of these
# functions stays below 10 in magnitude) and rounding 2^-52 |f| / H
DIFF_TOL = 10 * H * H + 2.0 ** -52 * 64 / H


def _rows(rng, rows, vocab):
    return rng.standard_normal((rows, vocab)) * 1.5


def _differences(f, z):
    g = np.empty_like(z)
    for r, j in np.ndindex(z.shape):
        up, down = z.copy(), z.copy()
        up[r, j] += H
        down[r, j] -= H
        g[r, j] = (f(up) - f(down)) / (2 * H)
    return g


@pytest.mark.parametrize("temperature", [0.7, 1.0, 2.0])
def test_logprob_gradient_equals_differences(temperature):
    rng = np.random.default_rng(3)
    z, tokens = _rows(rng, 4, 11), np.array([0, 10, -1, 5])
    gl, gh = rng.standard_normal(4), rng.standard_normal(4)

    def f(x):
        o = lm.token_logprobs(x, tokens, temperature)
        return float((gl * o["logprob"] + gh * o["entropy"])[tokens >= 0].sum())

    g, _ = lm.token_logprobs_backward(z, tokens, temperature, gl, gh)
    assert np.abs(g - _differences(f, z)).max() < DIFF_TOL


@pytest.mark.parametrize("temperature", [0.7, 1.0, 2.0])
def test_distill_gradient_equals_differences(temperature):
    rng = np.random.default_rng(4)
    z = _rows(rng, 4, 9)
    ids = np.array([[1, 4, 4], [8, -1, 0], [-1, -1, -1], [2, 3, 5]])  # an id twice, unused entries, an empty row
    teacher, w = rng.standard_normal((4, 3)) * 2, np.array([0.5, 1.0, 1.0, 0.25])
    _, _, g, _ = lm.distill_topk(z, ids, teacher, temperature, w)
    f = lambda x: float(lm.distill_topk(x, ids, teacher, temperature, w)[0].sum())  # noqa: E731
    assert np.abs(g - _differences(f, z)).max() < DIFF_TOL


def test_closed_forms():
    z = np.zeros((1, 8))
    o = lm.token_logprobs(z, [3], 1.0, top=3)
    assert o["logprob"][0] == pytest.approx(-math.log(8)) and o["entropy"][0] == pytest.approx(math.log(8))
    assert o["top_ids"][0].tolist() == [0, 1, 2]
    # the teacher equal to the student over the whole vocabulary: no loss, no gradient
    z = np.array([[0.5, -1.0, 2.0]])
    loss, _, g, _ = lm.distill_topk(z, [[2, 0, 1]], [[2.0, 0.5, -1.0]], 2.0)
    assert abs(loss[0]) < 1e-15 and np.abs(g).max() < 1e-15


def test_masked_rows():
    inf, nan = math.inf, math.nan
    z = np.array([[-inf, 1.0, -inf], [-inf, -inf, -inf], [0.0, nan, 0.0], [inf, 0.0, 0.0]])
    o = lm.token_logprobs(z, [1, 0, 0, 0], 1.0, top=2)
    assert o["logprob"][0] == 0 and o["entropy"][0] == 0 and o["top_ids"][0].tolist() == [1, 0]
    assert o["logprob"][1] == -inf and o["entropy"][1] == 0 and o["top_ids"][1].tolist() == [0, 1]
    assert np.isnan(o["logprob"][2:]).all() and (o["top_ids"][2:] == -1).all()
    g, _ = lm.token_logprobs_backward(z, [1, 0, 0, 0], 1.0, np.ones(4), np.ones(4))
    assert (g[:2] == 0).all() and np.isnan(g[2:]).all()


def test_codes_and_scales():
    # 2 ranks of 16 elements, blocks of 8: element j has scale (j // 16) * 2 + (j % 16) // 8
    codes = np.array([(i % 8) | ((8 + i % 8) << 4) for i in range(16)], np.uint8)
    scales = np.array([1, 2, 4, 8], np.float32)
    w = lm.quant_weights(codes, scales, 4, 8, 16, 2, 4, 7, 4)
    c = lm.decode_codes(codes, 4)
    assert c[:4].tolist() == [0, -8, 1, -7]
    assert w.reshape(-1).tolist() == [c[j] * float(scales[j // 8]) for j in range(4, 32)]
