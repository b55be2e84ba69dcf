"""The language-model operators as a training loop uses them around the step: a
head whose weights arrive by the quantized gather answers tokens (product,
log-probabilities with alternatives), is distilled from a teacher and pushed
by a policy gradient, and the weight gradients go through the shard step of
every rank into the next payload, from which the next tokens are answered.

Each hand-over is checked against the 64-bit oracle on what the operator
before it really delivered, so that errors cannot hide in one another.
"""
import math

import numpy as np
import pytest

import oracle
from oracle import lm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HIDDEN, VOCAB, N, BITS, BLOCK, ROWS, K = 256, 1003, 4, 4, 64, 24, 16


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


class Ranks:
    """The N ranks of one job on one device: state shards, and the gathered payload of their codes."""

    def __init__(self, zs, seed):
        import torch
        self.zs = zs
        self.plans = [zs.zs_shard_plan([HIDDEN, VOCAB * HIDDEN], N, r, BLOCK) for r in range(N)]
        self.S, self.T = self.plans[0].shard_numel, self.plans[0].padded_numel
        self.off = self.plans[0].tensor(1).flat_off
        gen = torch.Generator().manual_seed(seed)
        flat = torch.randn(self.T, generator=gen) * 0.05
        self.master = [flat[r * self.S:(r + 1) * self.S].clone().cuda() for r in range(N)]
        self.m = [torch.zeros(self.S, device="cuda") for _ in range(N)]
        self.v = [torch.zeros(self.S, device="cuda") for _ in range(N)]
        self.cb, self.ns = zs.zs_quant_code_bytes(self.plans[0], BITS), zs.zs_quant_num_scales(self.plans[0], BLOCK)
        self.codes = [torch.empty(self.cb, dtype=torch.uint8, device="cuda") for _ in range(N)]
        self.scales = [torch.empty(self.ns, device="cuda") for _ in range(N)]
        for r in range(N):
            zs.zs_quantize_shard(self.plans[r], BITS, BLOCK, self.master[r].bfloat16(), self.codes[r], self.scales[r])

    def payload(self):
        import torch
        return torch.cat(self.codes), torch.cat(self.scales)

    def weights(self):
        codes, scales = self.payload()
        return lm.quant_weights(codes.cpu().numpy(), scales.cpu().numpy(), BITS, BLOCK, self.S, self.ns, self.off,
                                VOCAB, HIDDEN)

    def answer(self, x):
        import torch
        codes, scales = self.payload()
        logits = torch.empty(x.shape[0], VOCAB, device="cuda")
        self.zs.zs_quant_matvec(self.plans[0], 1, VOCAB, HIDDEN, BITS, BLOCK, codes, scales, x, logits)
        return logits

    def step(self, grads, t):
        """grads: each rank's gradient of the whole flat buffer (bf16). Reduce, AdamW and codes of every shard."""
        hp = self.zs.AdamWHParams(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0, step=t)
        for r in range(N):
            own = [g[r * self.S:(r + 1) * self.S].clone() for g in grads]
            self.zs.zs_fused_shard_step_quant(self.plans[r], hp, own, self.master[r], self.m[r], self.v[r], BITS,
                                              BLOCK, self.codes[r], self.scales[r])
        return hp


def _check_logits(ranks, x, logits):
    ref, mag = lm.quant_matvec(ranks.weights(), x.double().cpu().numpy())
    assert (np.abs(logits.double().cpu().numpy() - ref) <= (HIDDEN + 2) * U * mag).all()


def test_answer_distill_step_answer(zs):
    import torch
    ranks = Ranks(zs, 0)
    gen = torch.Generator().manual_seed(1)
    rng = np.random.default_rng(2)
    ts = U * (VOCAB / 256 + 68 + 4 * math.log(VOCAB))
    xs = [torch.randn(ROWS, HIDDEN, generator=gen).bfloat16().cuda() for _ in range(N)]
    for t in (1, 2):
        grads = []
        for x in xs:  # every rank's micro-batch
            logits = ranks.answer(x)
            _check_logits(ranks, x, logits)
            host = logits.double().cpu().numpy()
            ids = np.array([rng.permutation(VOCAB)[:K] for _ in range(ROWS)])
            teacher = rng.standard_normal((ROWS, K)) * 2
            weight = np.full(ROWS, 1.0 / ROWS)
            weight[3] = 0.0  # a prompt position
            loss, d = torch.empty(ROWS, device="cuda"), torch.empty_like(logits)
            zs.zs_distill_topk(logits, torch.tensor(ids, dtype=torch.int32, device="cuda"),
                               torch.tensor(teacher, dtype=torch.float32, device="cuda"), loss, grad_logits=d,
                               temperature=2.0, row_weight=torch.tensor(weight, dtype=torch.float32, device="cuda"))
            t32 = teacher.astype(np.float32).astype(np.float64)
            w32 = weight.astype(np.float32).astype(np.float64)
            ref, lmag, g_ref, g_mag = lm.distill_topk(host, ids, t32, 2.0, w32)
            # exponentials of the teacher's and the student's differences (below 110) and their sums
            tol = 2 * ts + U * (K + 32 + 8 * 16)
            assert (np.abs(loss.cpu().numpy() - ref) <= tol * (lmag + 4 * w32 * math.log(VOCAB))).all()
            assert (np.abs(d.double().cpu().numpy() - g_ref) <= g_mag * tol + U * np.abs(g_ref)).all()
            # the policy gradient of the sampled tokens adds to it
            tokens = torch.tensor(rng.integers(0, VOCAB, ROWS), dtype=torch.int32, device="cuda")
            lp, stats = torch.empty(ROWS, device="cuda"), torch.empty(ROWS, 2, device="cuda")
            top = torch.empty(ROWS, 4, dtype=torch.int32, device="cuda")
            top_lp = torch.empty(ROWS, 4, device="cuda")
            zs.zs_token_logprobs(logits, tokens, logprob=lp, stats=stats, top_ids=top, top_logprobs=top_lp)
            scored = lm.token_logprobs(host, tokens.cpu().numpy(), 1.0, 4)
            assert np.array_equal(top.cpu().numpy(), scored["top_ids"])
            assert np.abs(lp.cpu().numpy() - scored["logprob"]).max() <= ts + 12 * U * np.abs(scored["logprob"]).max()
            advantage = torch.tensor(rng.standard_normal(ROWS) / ROWS, dtype=torch.float32, device="cuda")
            zs.zs_token_logprobs_backward(logits, tokens, stats, -advantage, logits)  # in place: the logits are spent
            pg, pg_mag = lm.token_logprobs_backward(host, tokens.cpu().numpy(), 1.0, -advantage.cpu().numpy())
            assert (np.abs(logits.double().cpu().numpy() - pg) <= pg_mag * (2 * ts + 200 * U) + U * np.abs(pg)).all()
            flat = torch.zeros(ranks.T, dtype=torch.bfloat16, device="cuda")
            flat[ranks.off:ranks.off + VOCAB * HIDDEN] = ((d + logits).t() @ x.float()).reshape(-1).bfloat16()
            grads.append(flat)
        before = [m.cpu().numpy().copy() for m in ranks.master], [m.cpu().numpy().copy() for m in ranks.m], \
            [v.cpu().numpy().copy() for v in ranks.v]
        hp = ranks.step(grads, t)
        for r in range(N):  # the step's own oracle takes the operators' gradients
            own = [g[r * ranks.S:(r + 1) * ranks.S].view(torch.int16).cpu().numpy().view(np.uint16) for g in grads]
            g16, p16 = np.zeros(ranks.S, np.uint16), np.zeros(ranks.S, np.uint16)
            full = np.zeros(ranks.T, np.uint16)
            oracle.shard_step(oracle.HParams(hp.lr, hp.beta1, hp.beta2, hp.eps, hp.weight_decay, t), own, g16,
                              before[0][r], before[1][r], before[2][r], p16, full, r)
            assert np.array_equal(before[0][r].view(np.uint32), ranks.master[r].cpu().numpy().view(np.uint32))
        changed = ranks.answer(xs[0])
        _check_logits(ranks, xs[0], changed)


def test_run_captured_in_a_graph(zs):
    """Answer, score and gradient captured as one graph and replayed on other inputs, eager work between the replays."""
    import torch
    ranks = Ranks(zs, 3)
    gen = torch.Generator().manual_seed(4)
    xs = [torch.randn(4, HIDDEN, generator=gen).bfloat16().cuda() for _ in range(3)]
    tokens = torch.tensor([5, -1, 900, 17], dtype=torch.int32, device="cuda")
    codes, scales = ranks.payload()

    class Out:
        def __init__(self):
            self.logits, self.g = torch.empty(4, VOCAB, device="cuda"), torch.empty(4, VOCAB, device="cuda")
            self.lp, self.en = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
            self.stats = torch.empty(4, 2, device="cuda")

        def go(self, x):
            zs.zs_quant_matvec(ranks.plans[0], 1, VOCAB, HIDDEN, BITS, BLOCK, codes, scales, x, self.logits)
            zs.zs_token_logprobs(self.logits, tokens, logprob=self.lp, entropy=self.en, stats=self.stats)
            zs.zs_token_logprobs_backward(self.logits, tokens, self.stats, self.lp, self.g, entropy=self.en,
                                          grad_entropy=self.en)

        def all(self):
            return [self.logits, self.g, self.lp, self.en, self.stats]

    want = []
    for x in xs:
        o = Out()
        o.go(x)
        want.append(o)
    static, out, eager = xs[0].clone(), Out(), Out()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.go(static)
    for i in (1, 2, 0, 2):
        static.copy_(xs[i])
        graph.replay()
        eager.go(xs[(i + 1) % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out.all(), want[i].all()))
        assert all(torch.equal(a, b) for a, b in zip(eager.all(), want[(i + 1) % 3].all()))
