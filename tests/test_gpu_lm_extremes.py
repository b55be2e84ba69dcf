"""Logits that lie farther apart than fp32's largest value, at temperatures that bring the quotient back into range.
Tolerances: log-probabilities and losses as test_gpu_lm_loss.py derives them, relative to values of this size."""
import numpy as np
import pytest

from test_gpu_lm_loss import _check_distill, _check_forward, _check_gradient, zs  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def _far_apart(vocab, dtype):
    import torch
    z = torch.full((5, vocab), -3e38)
    z[0, 3] = 3e38
    z[1] = torch.linspace(-3.3e38, 3.3e38, vocab)
    z[2, ::2] = 3e38
    z[3] = torch.randn(vocab, generator=torch.Generator().manual_seed(1)) * 1e38
    z[4] = -float("inf")
    z[4, 1], z[4, vocab - 1] = 3e38, -3e38
    return z.to(dtype).cuda()


@pytest.mark.parametrize("temperature", [1.0, 2.0, 2.5, 100.0, 1e6])
@pytest.mark.parametrize("vocab", [9, 5003, 40001])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_logprobs_of_logits_far_apart(zs, vocab, dtype, temperature):  # noqa: F811
    import torch
    z = _far_apart(vocab, getattr(torch, dtype))
    for tokens in ([0, 0, 1, 2, vocab - 1], [3, vocab - 1, 0, 1, 0], [vocab - 1, 1, 3, 0, 1]):
        _check_forward(zs, z, tokens, temperature, min(vocab, 7))
    _check_gradient(zs, z, [0, 0, 1, 2, vocab - 1], temperature, True)


@pytest.mark.parametrize("temperature", [1e-3, 0.5, 1.0, 2.5, 100.0, 1e3])
@pytest.mark.parametrize("vocab", [9, 5003, 70003])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_distillation_of_logits_far_apart(zs, vocab, dtype, temperature):  # noqa: F811
    import torch
    z = _far_apart(vocab, getattr(torch, dtype))
    ids = np.array([[0, 3, 5], [0, vocab - 1, 4], [1, 2, 3], [0, 1, 2], [1, vocab - 1, -1]])
    teacher = np.array([[1.0, 2.0, 0.0]] * 4 + [[3e38, 3e38, 0.0]])
    _check_distill(zs, z, ids, teacher, temperature)
