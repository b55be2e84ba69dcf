"""Log-probabilities of rows whose mask leaves a few tokens (answers bound to a grammar): fewer than, as many as and
more than the alternatives asked for, spread, side by side or among the first tokens. Tolerances are those of
test_gpu_lm_loss.py."""
import math

import numpy as np
import pytest

from test_gpu_lm_loss import _check_forward, _logits, zs  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu

COUNTS = (0, 1, 2, 9, 19, 20, 21, 31, 32, 33, 63, 64, 65, 200)


def _places(kind, n, vocab, rng):
    n = min(n, vocab)
    if kind == "spread":
        return rng.permutation(vocab)[:n]
    if kind == "first":
        return np.arange(n)
    if kind == "last":
        return vocab - 1 - np.arange(n)
    if kind == "every other of the first":
        return np.minimum(2 * np.arange(n), vocab - 1)
    start = int(rng.integers(0, vocab - n + 1))
    return start + np.arange(n)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [32, 40, 1003, 9000, 40001, 128256])
@pytest.mark.parametrize("kind", ["spread", "first", "last", "every other of the first", "side by side"])
def test_few_allowed_tokens(zs, kind, vocab, dtype):  # noqa: F811
    import torch
    rng = np.random.default_rng(vocab)
    counts = COUNTS if vocab < 100000 else COUNTS[::3]
    full = _logits(len(counts), vocab, dtype, seed=vocab)
    z = torch.full_like(full, -math.inf)
    tokens = []
    for r, n in enumerate(counts):
        at = _places(kind, n, vocab, rng)
        z[r, at] = full[r, at]
        if n > 3:  # equal ones and one of the type's lowest value among them
            z[r, at[1]] = z[r, at[2]]
            z[r, at[3]] = torch.finfo(z.dtype).min
        tokens.append(int(at[0]) if n and r % 2 else int(rng.integers(0, vocab)))
    z = z.cuda()
    for top in (1, 20, 32):
        _check_forward(zs, z, tokens, 0.8, top)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("threads", [256, 512])
def test_many_allowed_tokens_in_few_groups(zs, threads, dtype):  # noqa: F811
    """All of the allowed tokens lie in the vectors of a few threads: more than the list holds, in fewer groups than
    there are alternatives."""
    import torch
    vocab, wide = (8192, 8 if dtype == "bf16" else 4) if threads == 256 else (65536, 8 if dtype == "bf16" else 4)
    thread = torch.arange(vocab) // wide % threads
    full = _logits(4, vocab, dtype, seed=threads)
    z = torch.full_like(full, -math.inf)
    for r, most in enumerate((1, 9, 40, 80)):
        z[r, thread < most] = full[r, thread < most]
    _check_forward(zs, z.cuda(), [0, 1, vocab - 1, 5], 1.0, 20)
