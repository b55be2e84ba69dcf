"""Verification of drafted tokens with rows enough to fill the GPU, where waves sum pieces of 2048 logits (few rows:
of 512), against the same oracle and bounds as the small calls: 460 requests of 4 drafts are 4140 rows."""
import math

import numpy as np
import pytest

from test_gpu_drafts import Case, zs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

REQUESTS, K = 460, 4


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "certain"])
@pytest.mark.parametrize("vocab", [2049, 4096, 6151])
def test_matches_the_oracle(zs, vocab, dtype, with_draft):
    lens = np.random.default_rng(vocab).integers(-1, K + 2, REQUESTS)
    Case(zs, REQUESTS, K, vocab, dtype, vocab, with_draft, lens=lens, temperature=1.3, pad=5, shift=1).run()


@pytest.mark.parametrize("requests,k,vocab", [(341, 1, 2048), (2730, 1, 2048), (2731, 1, 2048), (8192, 0, 2047),
                                              (8191, 0, 7), (8193, 0, 1), (9000, 1, 513)])
def test_where_the_pieces_change(zs, requests, k, vocab):
    """8192 pieces are the border, and rows of 2048 logits: calls on either side."""
    Case(zs, requests, k, vocab, "f32", vocab).run()


def test_masks_nan_and_infinity(zs):
    for low in (-math.inf, -3.0e38):
        c = Case(zs, REQUESTS, K, 5003, "f32", 3)
        t, d = c.target.view(REQUESTS, K + 1, 5003), c.draft.view(REQUESTS, K, 5003)
        t[0] = low
        t[1, 1] = low
        t[2, 0, :-1] = low
        t[3, 0, 1:] = low
        t[4, 4, 2048:4096] = low
        d[5, 0] = low
        d[6, 1, :-1] = low
        t[7, 0, 4:] = low
        d[7, 0, 5:] = low
        t[8, 0, 2048:] = low
        d[8, 0, :2048] = low
        t[9, 0, :4096] = low
        t[10, 0, 77] = math.nan
        t[11, 2, 5002] = math.inf
        d[12, 0, 4096] = math.nan
        d[13, 3, 0] = math.inf
        c.tokens[2, 0] = 5002
        c.tokens[3, 0] = 17
        a = c.run()
        assert a[10] == 0 and a[12] == 0
        # a row of -infinity alone accepts nothing; the lowest values alone are 5003 tokens of like probability
        assert low > -math.inf or a[0] == 0


def test_borders(zs):
    """Rows of four equal likelihoods, one in each piece and one at the end: a random number on a border of the powers
    of two belongs to the token behind it."""
    vocab, places = 8192, (5, 2048, 4099, 8191)
    c = Case(zs, 2100, 0, vocab, "f32", 4)
    c.target.fill_(-math.inf)
    for j in places:
        c.target[:, j] = 1.5
    c.uniforms[:, 0] = np.arange(2100) % 8 / 8
    c.run()
    assert c.out[1].view(-1).tolist() == [places[i % 8 // 2] for i in range(2100)]


def test_a_workspace_serves_smaller_calls(zs):
    """The workspace of the largest call, given whole to smaller ones on both sides of the border."""
    big = Case(zs, REQUESTS, K, 6151, "bf16", 6).device()
    for requests, k, vocab in ((1, 4, 6151), (460, 4, 500), (117, 3, 6151), (459, 4, 6151), (240, 4, 3001)):
        assert zs.zs_verify_drafts_workspace_bytes(requests, k, vocab) <= big.need
        c = Case(zs, requests, k, vocab, "f32", 7).device()
        c.work, c.need = big.work, big.need
        c.call()
        c.check()
    big.call()
    big.check()


def test_equal_bits_in_a_graph_and_on_another_stream(zs):
    import torch
    c = Case(zs, REQUESTS, K, 5003, "bf16", 8).device()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    c.call(side)
    c.check()
    held = [o.clone() for o in c.out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call()
    for _ in range(3):
        for o in c.out:
            o.fill_(5)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, c.out))
        c.call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, c.out))
