"""Verification of drafted tokens on the GPU against the 64-bit oracle: tokens and counts have to be equal (random
numbers lie on no border of either), log-probabilities within an fp32 rounding (2^-24 relative, and the error of 64-bit
sums, far below)."""
import math

import numpy as np
import pytest

from oracle import drafts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


class Case:
    """Inputs of a call on the GPU and as float64, its outputs with a guard behind each."""

    def __init__(self, zs, requests, k, vocab, dtype, seed, with_draft=True, lens=None, temperature=1.0, pad=0,
                 spread=2.0, shift=0):
        import torch
        self.zs, self.t, self.k = zs, temperature, k
        rng = np.random.default_rng(seed)
        kind = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]

        def logits(rows, values):
            base = torch.zeros(max(rows - 1, 0) * (vocab + pad) + vocab + shift, dtype=kind, device="cuda")
            m = base[shift:].as_strided((rows, vocab), (vocab + pad, 1))
            m.copy_(torch.from_numpy(values.reshape(rows, vocab).astype(np.float32)))
            return m

        target = rng.standard_normal((requests, k + 1, vocab)) * spread
        for row in target.reshape(-1, vocab):
            row[rng.integers(0, vocab, 4)] += 6
        self.target = logits(requests * (k + 1), target)
        self.draft = logits(requests * k, target[:, :k] + 0.7 * rng.standard_normal((requests, k, vocab))) \
            if with_draft and k else None
        self.tokens = np.zeros((requests, k), np.int32)
        drawn_from = self.draft64() if self.draft is not None else target
        for b in range(requests):
            for i in range(k):
                p = drafts.softmax(drawn_from[b, i], temperature)
                self.tokens[b, i] = np.searchsorted(np.cumsum(p), rng.random() * p.sum()).clip(0, vocab - 1)
        self.uniforms = rng.random((requests, k + 1)).astype(np.float32)
        self.lens = None if lens is None else np.asarray(lens, np.int32)

    def target64(self):
        return self.target.double().cpu().numpy().reshape(-1, self.k + 1, self.target.shape[1])

    def draft64(self):
        return None if self.draft is None else self.draft.double().cpu().numpy().reshape(-1, self.k,
                                                                                        self.target.shape[1])

    def device(self):
        import torch
        requests, k, vocab = len(self.tokens), self.k, self.target.shape[1]
        self.d = dict(tokens=torch.from_numpy(self.tokens).cuda(), uniforms=torch.from_numpy(self.uniforms).cuda(),
                      lens=None if self.lens is None else torch.from_numpy(self.lens).cuda())
        self.guard = [torch.full((requests + 8,), 77, dtype=torch.int32, device="cuda"),
                      torch.full((requests * (k + 1) + 8,), 77, dtype=torch.int32, device="cuda"),
                      torch.full((requests * (k + 1) + 8,), 77.0, device="cuda")]
        need = self.zs.zs_verify_drafts_workspace_bytes(requests, k, vocab)
        self.work = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN, were it read
        self.out = (self.guard[0][:requests], self.guard[1][:-8].view(requests, k + 1),
                    self.guard[2][:-8].view(requests, k + 1))
        self.need = need
        return self

    def call(self, stream=None):
        self.zs.zs_verify_drafts(self.target, self.d["tokens"], self.d["uniforms"], self.out[0], self.out[1],
                                 self.work[:self.need], draft_logits=self.draft, draft_lens=self.d["lens"],
                                 logprobs=self.out[2], temperature=self.t, stream=stream)

    def check(self):
        import torch
        torch.cuda.synchronize()
        a, t, lp = drafts.verify(self.target64(), self.draft64(), self.tokens, self.lens, self.uniforms, self.t)
        assert np.array_equal(self.out[0].cpu().numpy(), a)
        assert np.array_equal(self.out[1].cpu().numpy(), t)
        got = self.out[2].double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(lp))
        fine = ~np.isnan(lp)
        assert (np.abs(got - lp)[fine] <= 2.0 ** -24 * np.abs(lp[fine]) + 1e-12).all()
        assert all(bool((g[-8:] == 77).all()) for g in self.guard)
        assert bool((self.work[self.need:] == 0xFF).all())
        return a

    def run(self):
        self.device().call()
        return self.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("with_draft", [True, False], ids=["draft", "certain"])
@pytest.mark.parametrize("requests,k,vocab", [(1, 1, 1), (1, 4, 3), (2, 3, 100), (5, 4, 1003), (3, 2, 8191),
                                              (3, 2, 8192), (3, 2, 8193), (2, 5, 16385), (4, 8, 32000), (1, 64, 515),
                                              (40, 1, 257), (300, 2, 33)])
def test_matches_the_oracle(zs, requests, k, vocab, dtype, with_draft):
    Case(zs, requests, k, vocab, dtype, requests + vocab, with_draft, temperature=0.8).run()


def test_large_vocabulary_and_flat_rows(zs):
    """151936 tokens of nearly like probability: borders 7e-6 apart, over 40 requests."""
    c = Case(zs, 40, 2, 151936, "f32", 1, spread=0.01)
    a = c.run()
    assert (a < 2).any() and (a == 2).any()


@pytest.mark.parametrize("k", [0, 3])
def test_strides_and_alignment(zs, k):
    for dtype in ("bf16", "f32"):
        for pad, shift in ((1, 1), (5, 3), (24, 0)):
            Case(zs, 3, k, 1001, dtype, pad, pad=pad, shift=shift).run()


def test_no_drafts_draws_from_each_row(zs):
    c = Case(zs, 20, 0, 5000, "bf16", 4)
    assert not c.run().any()


@pytest.mark.parametrize("lens", [[0, 1, 2, 3, 4, 9, -1, -5], [4] * 8, [-1] * 8, [0] * 8])
def test_lengths(zs, lens):
    """Short, full, too long and skipped requests; what lies behind a request's rows is not looked at."""
    for with_draft in (True, False):
        c = Case(zs, 8, 4, 700, "f32", 6, with_draft, lens=lens)
        for b, n in enumerate(lens):
            for i in range(max(n + 1, 0), 5):
                c.target[b * 5 + i] = math.nan
            for i in range(max(n, 0), 4):
                if with_draft:
                    c.draft[b * 4 + i] = math.inf
                c.tokens[b, i] = -(1 << 31)
        c.run()


def test_equal_models_accept_everything(zs):
    c = Case(zs, 16, 6, 3000, "bf16", 9)
    c.draft.copy_(c.target.view(16, 7, 3000)[:, :6].reshape(96, 3000))
    c.uniforms[:, :6] = 1 - 2.0 ** -24
    assert (c.run() == 6).all()


def test_masks(zs):
    """Rows that leave one token, few, or none; draft rows that leave none; the type's lowest value instead."""
    for low in (-math.inf, -3.0e38):
        c = Case(zs, 12, 3, 9000, "f32", 11)
        t, d = c.target.view(12, 4, 9000), c.draft.view(12, 3, 9000)
        t[0, :, :] = low
        t[1, 1, :] = low
        t[2, 0, :-1] = low
        t[3, 0, 1:] = low
        t[4, 3, 5:8990] = low
        d[5, 0, :] = low
        d[6, 1, :-1] = low
        t[7, 0, 4:] = low
        d[7, 0, 5:] = low
        t[8, 2, 8192:] = low
        t[9, 0, :8192] = low
        c.tokens[2, 0] = 8999
        c.tokens[3, 0] = 17  # masked in the target: falls
        c.run()


def test_nan_and_infinity(zs):
    for bad in (math.nan, math.inf):
        c = Case(zs, 8, 3, 8200, "bf16", 13)
        t, d = c.target.view(8, 4, 8200), c.draft.view(8, 3, 8200)
        t[0, 0, 8199] = bad
        t[1, 1, 0] = bad
        t[2, 3, 77] = bad
        d[3, 0, 5] = bad
        d[4, 2, 8192] = bad
        t[5, :, 1] = bad
        d[6, :, 1] = bad
        c.uniforms[:, :3] = 0.05
        a = c.run()
        assert a[0] == 0 and a[3] == 0


def test_tokens_outside_the_vocabulary_fall(zs):
    for with_draft in (True, False):
        c = Case(zs, 6, 2, 500, "f32", 15, with_draft)
        c.tokens[:, 0] = [-1, 500, (1 << 31) - 1, -(1 << 31), 3, 499]
        c.uniforms[:, 0] = 0
        a = c.run()
        assert not a[:4].any()


def test_borders_and_odd_random_numbers(zs):
    """Powers of two are exact: a random number on a border belongs to the token behind it. Numbers at and above 1,
    below 0 and NaN draw the last and the first token that has a probability."""
    import torch
    vocab = 8192 * 2
    c = Case(zs, 12, 0, vocab, "f32", 17)
    c.target.fill_(0.0)
    c.target[6:].fill_(-math.inf)
    c.target[6:, 100:100 + 64] = 0.0
    c.uniforms[:, 0] = [0, 1 / vocab, 0.5, 8191 / vocab, 1 - 2.0 ** -24, 1.0, 0, 1 / 64, 0.5, 2.0, -1.0, math.nan]
    c.device().call()
    torch.cuda.synchronize()
    want = [0, 1, 8192, 8191, 16383, 16383, 100, 101, 132, 163, 100, 100]
    assert c.out[1][:, 0].tolist() == want
    c.check()
    # a token of probability 1/8 that the draft was certain of stands below 1/8 and falls on it
    c = Case(zs, 3, 1, 8, "f32", 18, with_draft=False)
    c.target.fill_(1.0)
    c.tokens[:] = 5
    c.uniforms[:] = [[0.125, 0.0], [0.125 - 2.0 ** -27, 0.0], [math.nan, 0.99]]
    assert c.run().tolist() == [0, 1, 0]


@pytest.mark.parametrize("temperature", [1e-6, 0.05, 1.0, 50.0, 1e6])
def test_temperatures(zs, temperature):
    Case(zs, 6, 3, 9001, "f32", 21, temperature=temperature).run()
    Case(zs, 6, 3, 1001, "bf16", 21, temperature=temperature).run()


def test_without_logprobs_and_with_more_workspace(zs):
    import torch
    c = Case(zs, 4, 3, 1000, "f32", 23).device()
    c.call()
    tokens = c.out[1].clone()
    c.out[1].fill_(77)
    zs.zs_verify_drafts(c.target, c.d["tokens"], c.d["uniforms"], c.out[0], c.out[1], c.work, draft_logits=c.draft)
    torch.cuda.synchronize()
    assert torch.equal(tokens, c.out[1])


def test_streams_and_shared_workspace_in_graphs(zs):
    """Two captured calls that share a workspace, replayed one after the other on one stream, with eager calls
    between."""
    import torch
    a, b = Case(zs, 6, 4, 20000, "f32", 31).device(), Case(zs, 3, 2, 9000, "bf16", 32).device()
    b.work = a.work
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(side)
    a.check()
    graphs = []
    for c in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.call()
        graphs.append(g)
    rng = np.random.default_rng(5)
    for _ in range(3):
        for c in (a, b):
            c.uniforms[:] = rng.random(c.uniforms.shape)
            c.d["uniforms"].copy_(torch.from_numpy(c.uniforms))
            c.out[1].fill_(5)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        for c in (a, b):
            need, c.need = c.need, c.work.numel() - 64 if c is b else c.need
            c.check()
            c.need = need
        b.call()
        b.need, need = b.work.numel() - 64, b.need
        b.check()
        b.need = need


def test_binding_refusals(zs):
    import torch
    c = Case(zs, 3, 2, 100, "f32", 41).device()
    good = dict(target_logits=c.target, draft_tokens=c.d["tokens"], uniforms=c.d["uniforms"], accepted=c.out[0],
                tokens=c.out[1], workspace=c.work[:c.need], draft_logits=c.draft, logprobs=c.out[2])
    for bad in (dict(target_logits=c.target[:8]), dict(draft_tokens=c.d["tokens"].long()),
                dict(uniforms=c.d["uniforms"][:, :2]), dict(accepted=c.out[0][:2]), dict(tokens=c.out[1][:, :2]),
                dict(draft_logits=c.draft.bfloat16()), dict(draft_logits=c.draft[:5]), dict(logprobs=c.out[2].double()),
                dict(draft_lens=torch.zeros(2, dtype=torch.int32, device="cuda")),
                dict(target_logits=c.target.cpu()), dict(draft_tokens=c.d["tokens"].cpu())):
        with pytest.raises(ValueError):
            zs.zs_verify_drafts(**dict(good, **bad))
    with pytest.raises(zs.ZsError):
        zs.zs_verify_drafts(**dict(good, workspace=c.work[:c.need - 1]))
    with pytest.raises(zs.ZsError):
        zs.zs_verify_drafts(**dict(good, temperature=0.0))
