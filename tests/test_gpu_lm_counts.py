"""Log-probabilities with every count of equal best logits around the sizes of the list that ranks them, and rows whose
thread count changes with their length; distillation with the most entries a row takes, in workgroups of every size.
Tolerances are those of test_gpu_lm_loss.py."""
import numpy as np
import pytest

from test_gpu_lm_loss import _check_distill, _check_forward, _logits, _teacher, zs  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [600, 5001, 40001])
def test_counts_of_equal_best_logits(zs, vocab, dtype):  # noqa: F811
    """The lowest tokens among the equal ones come first, whether one wave, the block or rounds rank them."""
    counts = [1, 2, 31, 32, 33, 63, 64, 65, 100, 128, 255, 256, 257, 300, 400, 511, 512, 513, 600]
    z = _logits(len(counts), vocab, dtype, seed=vocab)
    rng = np.random.default_rng(vocab)
    for r, n in enumerate(counts):
        z[r, rng.permutation(vocab)[:n].tolist()] = 20.0
    z = z.cuda()
    for top in (1, 20, 32):
        _check_forward(zs, z, rng.integers(0, vocab, len(counts)).tolist(), 1.0, top)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 65535), ("bf16", 65536), ("f32", 24575), ("f32", 24576)])
def test_many_rows_around_the_length_that_takes_more_threads(zs, vocab, dtype):  # noqa: F811
    import torch
    rows = 1027
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device="cuda")
    at = [0, 513, rows - 1]
    part = _logits(len(at), vocab, dtype, seed=9).cuda()
    z[at] = part
    tokens = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    tokens[at] = torch.tensor([1, vocab // 2, vocab - 1], dtype=torch.int32, device="cuda")
    out = {"logprob": torch.empty(rows, device="cuda"), "entropy": torch.empty(rows, device="cuda"),
           "stats": torch.empty(rows, 2, device="cuda"), "top_ids": torch.empty(rows, 9, dtype=torch.int32, device="cuda"),
           "top_logprobs": torch.empty(rows, 9, device="cuda")}
    zs.zs_token_logprobs(z, tokens, **out)
    # the same rows alone: within the tolerance of both (fewer rows may take other threads)
    few, _ = _check_forward(zs, part, [1, vocab // 2, vocab - 1], 1.0, 9)
    assert torch.equal(out["top_ids"][at], few.out["top_ids"])
    for name in ("logprob", "entropy", "stats", "top_logprobs"):
        # two results that are each within a few hundred units of 2^-24 of the same value below 32
        assert (out[name][at] - few.out[name]).abs().max().item() <= 2 * 2000 * 2.0 ** -24 * 32, name
        skipped = torch.ones(rows, dtype=torch.bool, device="cuda")
        skipped[at] = False
        assert not out[name][skipped].any()
    assert (out["top_ids"][tokens < 0] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1500, 9001, 30011, 61003, 140001])
def test_distillation_with_the_most_entries(zs, vocab, dtype):  # noqa: F811
    rng = np.random.default_rng(vocab)
    ids, teacher = _teacher(rng, 5, 1024, vocab)
    ids[1, 512:] = ids[1, :512]              # every token twice
    ids[2, :] = 7                            # one token
    ids[3, 1::2] = -1
    ids[4, -1] = ids[4, 0]                   # the last entry repeats the first
    _check_distill(zs, _logits(5, vocab, dtype, seed=vocab).cuda(), ids, teacher, 1.3, [1.0, 0.5, 2.0, -1.0, 1.0])
