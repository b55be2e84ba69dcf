"""The verification of drafted tokens at the largest vocabulary and with the most requests that it takes."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


def test_the_largest_vocabulary(zs):
    """2^30 logits a row, all masked but three of like probability: in the first piece, past the middle and the last."""
    import torch
    vocab = 1 << 30
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GiB")
    target = torch.full((2, vocab), -math.inf, dtype=torch.bfloat16, device="cuda")
    three = [5, (1 << 29) + 7, vocab - 1]
    target[:, three] = 1.0
    work = torch.empty(zs.zs_verify_drafts_workspace_bytes(1, 1, vocab), dtype=torch.uint8, device="cuda")
    accepted = torch.empty(1, dtype=torch.int32, device="cuda")
    out = torch.empty(1, 2, dtype=torch.int32, device="cuda")
    lp = torch.empty(1, 2, device="cuda")
    third = -math.log(3.0)
    # the drafted token, the random numbers, and what comes out: tokens and how many have a log-probability
    for x, u0, u1, want in ((three[2], 0.25, 0.5, [three[2], three[1]]), (three[1], 0.25, 0.9, [three[1], three[2]]),
                            (three[2], 0.5, 0.4, [three[0], -1]), (three[2], 0.5, 0.9, [three[1], -1]),
                            (three[0], 0.75, 0.75, [three[2], -1]), (6, 0.0, 0.0, [three[0], -1])):
        tokens = torch.tensor([[x]], dtype=torch.int32, device="cuda")
        zs.zs_verify_drafts(target, tokens, torch.tensor([[u0, u1]], device="cuda"), accepted, out, work, logprobs=lp)
        assert out.tolist() == [want] and int(accepted) == (want[1] >= 0)
        for t, v in zip(want, lp[0].tolist()):
            assert v == 0.0 if t < 0 else abs(v - third) <= 2.0 ** -24 * abs(third) + 1e-12


def test_the_most_requests(zs):
    """A token drawn from each of 2^22 - 1 rows of three logits. A draw is compared where the random number is farther
    from a border than 64-bit sums of three can be off."""
    import torch
    requests, vocab = (1 << 22) - 1, 3
    torch.manual_seed(3)
    target = torch.randn(requests, vocab, device="cuda") * 3
    u = torch.rand(requests, 1, device="cuda")
    work = torch.empty(zs.zs_verify_drafts_workspace_bytes(requests, 0, vocab), dtype=torch.uint8, device="cuda")
    accepted = torch.full((requests,), 7, dtype=torch.int32, device="cuda")
    out = torch.full((requests, 1), 7, dtype=torch.int32, device="cuda")
    zs.zs_verify_drafts(target, torch.empty(requests, 0, dtype=torch.int32, device="cuda"), u, accepted, out, work)
    z = target.double().cpu().numpy()
    e = np.exp(z - z.max(axis=1, keepdims=True))
    run = np.cumsum(e, axis=1)
    border = u.double().cpu().numpy() * run[:, -1:]
    want = (run <= border).sum(axis=1)
    clear = (np.abs(run - border) > 1e-13).all(axis=1)
    assert clear.mean() > 0.999
    assert np.array_equal(out.cpu().numpy()[clear, 0], want[clear])
    assert not bool(accepted.any())
    with pytest.raises(zs.ZsError):
        zs.zs_verify_drafts_workspace_bytes(requests + 1, 0, vocab)
