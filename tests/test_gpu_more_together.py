"""The 4-bit format, the verification of drafted tokens and the clipped multi-tensor step as a training loop with
sampled rollouts uses them: every rank's wrapped pieces are reduced, their norm clips the step, the gathered head is
quantized, the head of the step before drafts tokens and the new one verifies them, and the next gradients follow.

Each hand-over is checked against the oracle on what the operator before it really delivered, so that errors cannot
hide in one another. Products of `blocks` 32-column blocks are within (ceil(blocks / 2) + 16) 2^-21 of the sum of
magnitudes: an fp32 sum of as many 64-column steps and of at most 16 waves' parts, each an instruction whose own sum
of 64 products is off by up to 2^-21 of theirs."""
import numpy as np
import pytest

import oracle
from gpu_util import dev16, dev32, host16, host32
from oracle import drafts, mx4

pytestmark = pytest.mark.gpu

HIDDEN, VOCAB, N, REQUESTS, K = 200, 1003, 4, 6, 3
NUMELS = [VOCAB * HIDDEN, HIDDEN, 5]
MAX_NORM = 0.5


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


class Ranks:
    """The N ranks of one job on one device. The gathered tensors are shared: every rank writes its own part."""

    def __init__(self, zs, seed):
        import torch
        self.zs = zs
        self.rng = np.random.default_rng(seed)
        self.plans = [zs.zs_shard_plan_ex(NUMELS, N, r, persist_below_elems=300) for r in range(N)]
        infos = [[p.tensor(i) for i in range(len(NUMELS))] for p in self.plans]
        self.padded = [i.padded_numel for i in infos[0]]
        self.own = [[(i.own_lo, i.own_hi) for i in info] for info in infos]
        self.replicated = [zs.lib().zs_plan_tensor_replicated(self.plans[0].handle, i) for i in range(len(NUMELS))]
        assert self.replicated == [0, 1, 1]
        whole = [np.zeros(n, np.float32) for n in self.padded]
        for w, n in zip(whole, NUMELS):
            w[:n] = self.rng.standard_normal(n) * 0.3
        self.full = [dev16(oracle.f32_to_bf16(w)) for w in whole]
        self.o, self.d, self.ws, self.grads = [], [], [], []
        self.sumsq = torch.zeros(N, dtype=torch.float64, device="cuda")
        self.flags = torch.zeros(N, dtype=torch.int32, device="cuda")
        for r, plan in enumerate(self.plans):
            o = [dict(master=w[lo:hi].copy(), m=np.zeros(hi - lo, np.float32), v=np.zeros(hi - lo, np.float32),
                      p=np.zeros(hi - lo, np.uint16)) for w, (lo, hi) in zip(whole, self.own[r])]
            d = [dict(grad=dev16(np.zeros(x["p"].size, np.uint16)), master=dev32(x["master"]), m=dev32(x["m"]),
                      v=dev32(x["v"]), param=dev16(x["p"]), full=f) for x, f in zip(o, self.full)]
            grads = [[torch.zeros_like(x["grad"]) for x in d] for _ in range(N)]
            ws = torch.zeros(zs.zs_multi_workspace_bytes(plan, N), dtype=torch.uint8, device="cuda")
            zs.zs_multi_bind(plan, d, grads, ws)
            self.o.append(o)
            self.d.append(d)
            self.ws.append(ws)
            self.grads.append(grads)
        self.stats = torch.empty(max(zs.zs_grad_stats_multi_workspace_bytes(p) for p in self.plans),
                                 dtype=torch.uint8, device="cuda")
        self.scale = torch.empty(1, device="cuda")
        self.skip = torch.empty(1, dtype=torch.int32, device="cuda")

    def step(self, step, size, bad=None):
        """Gradients of every rank, their average, its norm over all ranks and the clipped step."""
        import torch
        zs = self.zs
        whole = [[np.zeros(n, np.uint16) for n in self.padded] for _ in range(N)]
        for q in range(N):
            for i, n in enumerate(NUMELS):
                whole[q][i][:n] = oracle.f32_to_bf16(np.float32(self.rng.standard_normal(n) * size))
        if bad is not None:
            whole[1][0][bad] = 0x7F80
        hp = zs.AdamWHParams(lr=2e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=step)
        for r, plan in enumerate(self.plans):
            for q in range(N):
                for i, (lo, hi) in enumerate(self.own[r]):
                    self.grads[r][q][i].copy_(dev16(whole[q][i][lo:hi]))
            zs.zs_reduce_shard_multi(plan, self.ws[r])
            zs.zs_grad_stats_multi(plan, self.sumsq[r:], self.flags[r:], self.ws[r], self.stats)
        zs.zs_clip_scale(self.sumsq, self.flags, MAX_NORM, self.scale, self.skip)
        for r, plan in enumerate(self.plans):
            zs.zs_adamw_shard_step_multi_clip(plan, [hp], self.ws[r], scale=self.scale, skip=self.skip)
        torch.cuda.synchronize()
        total, count = 0.0, 0
        for r in range(N):
            for i, (lo, hi) in enumerate(self.own[r]):
                g = oracle.reduce([whole[q][i][lo:hi].copy() for q in range(N)]) if hi > lo else np.zeros(0, np.uint16)
                assert np.array_equal(host16(self.d[r][i]["grad"]), g)
                if not (self.replicated[i] and r) and g.size:
                    total += oracle.grad_sumsq(oracle.bf16_to_f32(g))[0]
                    count += g.size
        sums = self.sumsq.cpu().numpy()
        if bad is not None:
            assert int(self.skip) == 1
        else:
            assert int(self.skip) == 0 and abs(sums.sum() - total) <= (count + N) * 2.0 ** -53 * total
            want = np.float32(oracle.clip_scale(list(sums), MAX_NORM))
            assert np.float32(self.scale.item()) == want and (want < 1.0) == (total > MAX_NORM ** 2)
            for r in range(N):
                for o, d in zip(self.o[r], self.d[r]):
                    if o["p"].size:
                        oracle.adamw_f32grad(oracle.HParams(2e-2, 0.9, 0.95, 1e-8, 0.1, step),
                                             oracle.bf16_to_f32(host16(d["grad"])), 1.0, float(want), 0, o["master"],
                                             o["m"], o["v"], o["p"])
        for r in range(N):
            for i, (o, d) in enumerate(zip(self.o[r], self.d[r])):
                for name in ("master", "m", "v"):
                    assert np.array_equal(host32(d[name]).view(np.uint32), o[name].view(np.uint32)), (r, i, name)
                assert np.array_equal(host16(d["param"]), o["p"])
                lo, hi = self.own[r][i]
                if bad is None:
                    assert np.array_equal(host16(self.full[i])[lo:hi], o["p"])

    def head(self):
        """Codes and scales of the gathered head, and their values."""
        import torch
        w = self.full[0][:NUMELS[0]].view(torch.bfloat16).view(VOCAB, HIDDEN)
        return _quantized(self.zs, w)

    def close(self):
        for ws in self.ws:
            self.zs.zs_multi_unbind(ws)


def _quantized(zs, x):
    import torch
    rows, cols = x.shape
    blocks = -(-cols // 32)
    codes = torch.empty(rows, 16 * blocks, dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows, blocks, dtype=torch.uint8, device="cuda")
    zs.zs_mx4_quantize(x, codes, scales)
    want = mx4.quantize(x[:8].double().cpu().numpy())  # the oracle takes element by element
    assert np.array_equal(codes[:8].cpu().numpy(), want[0]) and np.array_equal(scales[:8].cpu().numpy(), want[1])
    back = torch.empty(rows, cols, device="cuda")
    zs.zs_mx4_dequantize(codes, scales, back)
    values = mx4.dequantize(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(back.double().cpu().numpy(), values[:, :cols]) and not values[:, cols:].any()
    return codes, scales, values


def _logits(zs, x, head):
    import torch
    codes, scales, values = _quantized(zs, x)
    y = torch.empty(x.shape[0], VOCAB, device="cuda")
    zs.zs_mx4_matmul(codes, scales, head[0], head[1], y)
    want, mag = mx4.matmul(values, head[2])
    blocks = -(-HIDDEN // 32)
    assert (np.abs(y.double().cpu().numpy() - want) <= (-(-blocks // 2) + 16) * 2.0 ** -21 * mag).all()
    return y


def _verify(zs, target, tokens, uniforms, **kw):
    import torch
    requests, places = uniforms.shape
    out = (torch.empty(requests, dtype=torch.int32, device="cuda"),
           torch.empty(requests, places, dtype=torch.int32, device="cuda"),
           torch.empty(requests, places, device="cuda"))
    work = torch.empty(zs.zs_verify_drafts_workspace_bytes(requests, places - 1, VOCAB), dtype=torch.uint8,
                       device="cuda")
    zs.zs_verify_drafts(target, tokens, uniforms, out[0], out[1], work, logprobs=out[2], temperature=0.9, **kw)
    shaped = {"lens": kw.get("draft_lens"), "draft": kw.get("draft_logits")}
    a, t, lp = drafts.verify(target.double().cpu().numpy().reshape(requests, places, VOCAB),
                             None if shaped["draft"] is None else
                             shaped["draft"].double().cpu().numpy().reshape(requests, places - 1, VOCAB),
                             tokens.cpu().numpy(), None if shaped["lens"] is None else shaped["lens"].cpu().numpy(),
                             uniforms.cpu().numpy(), 0.9)
    assert np.array_equal(out[0].cpu().numpy(), a) and np.array_equal(out[1].cpu().numpy(), t)
    assert (np.abs(out[2].double().cpu().numpy() - lp) <= 2.0 ** -24 * np.abs(lp) + 1e-12).all()
    return out


def test_step_quantize_draft_verify(zs):
    import torch
    ranks = Ranks(zs, 0)
    gen = torch.Generator(device="cuda").manual_seed(1)
    old = ranks.head()
    seen = set()
    for step in (1, 2, 3):
        if step == 2:  # a gradient that is not finite leaves state and head as they are
            before = ranks.full[0].clone()
            ranks.step(step, 1e-3, bad=77)
            assert torch.equal(before, ranks.full[0])
        ranks.step(step, 1e-2 if step == 1 else 1e-4)
        new = ranks.head()
        hidden = torch.randn(REQUESTS, K + 1, HIDDEN, device="cuda", generator=gen)
        gain = ranks.full[1].view(torch.bfloat16).float()
        x = (hidden * (1.0 + gain)).to(torch.bfloat16)
        drafted = _logits(zs, x[:, :K].reshape(-1, HIDDEN), old)
        empty = torch.empty(REQUESTS * K, 0, dtype=torch.int32, device="cuda")
        u = torch.rand(REQUESTS * K, 1, device="cuda", generator=gen)
        tokens = _verify(zs, drafted, empty, u)[1].view(REQUESTS, K)  # no drafts: a token of each row
        target = _logits(zs, x.view(-1, HIDDEN), new)
        lens = torch.tensor([K, K, 1, 0, -1, K + 2], dtype=torch.int32, device="cuda")
        u = torch.rand(REQUESTS, K + 1, device="cuda", generator=gen)
        accepted, out, lps = _verify(zs, target, tokens, u, draft_logits=drafted, draft_lens=lens)
        for n, row in zip(accepted.tolist(), out.tolist()):
            seen.add(n)
            assert all(t >= 0 for t in row[:n]) and all(t == -1 for t in row[n + 1:])
        # the accepted tokens' log-probabilities are the language-model operator's at that temperature
        flat = torch.empty(target.shape[0], device="cuda")
        zs.zs_token_logprobs(target, out.view(-1).clamp(min=0), logprob=flat, temperature=0.9)
        kept = out.view(-1) >= 0
        # the operator's own bound for rows of VOCAB logits: exponentials and their sum in fp32
        tol = 2.0 ** -24 * (VOCAB / 256 + 68 + 4 * np.log(VOCAB)) + 13 * 2.0 ** -24 * lps.view(-1).abs()
        assert bool(((flat - lps.view(-1)).abs() <= tol)[kept].all())
        old = new
    ranks.close()
    assert len(seen) > 1


def test_captured_round_follows_its_inputs(zs):
    """Norm, factor, clipped step, quantization, products and verification captured as one graph, replayed with new
    gradients, hidden states and random numbers between eager work, against the same calls made eagerly."""
    import torch
    pair = [Ranks(zs, 5), Ranks(zs, 5)]
    blocks = -(-HIDDEN // 32)

    def u8(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device="cuda")

    bufs = [dict(wc=u8(VOCAB, 16 * blocks), ws=u8(VOCAB, blocks), xc=u8(REQUESTS * (K + 1), 16 * blocks),
                 xs=u8(REQUESTS * (K + 1), blocks), y=torch.empty(REQUESTS * (K + 1), VOCAB, device="cuda"),
                 accepted=torch.empty(REQUESTS, dtype=torch.int32, device="cuda"),
                 out=torch.empty(REQUESTS, K + 1, dtype=torch.int32, device="cuda"),
                 lps=torch.empty(REQUESTS, K + 1, device="cuda"),
                 work=u8(zs.zs_verify_drafts_workspace_bytes(REQUESTS, K, VOCAB))) for _ in pair]
    x = torch.empty(REQUESTS * (K + 1), HIDDEN, dtype=torch.bfloat16, device="cuda")
    tokens = torch.empty(REQUESTS, K, dtype=torch.int32, device="cuda")
    u = torch.empty(REQUESTS, K + 1, device="cuda")
    hp = zs.AdamWHParams(lr=2e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=4)

    def calls(ranks, b):
        for r, plan in enumerate(ranks.plans):
            zs.zs_reduce_shard_multi(plan, ranks.ws[r])
            zs.zs_grad_stats_multi(plan, ranks.sumsq[r:], ranks.flags[r:], ranks.ws[r], ranks.stats)
        zs.zs_clip_scale(ranks.sumsq, ranks.flags, MAX_NORM, ranks.scale, ranks.skip)
        for r, plan in enumerate(ranks.plans):
            zs.zs_adamw_shard_step_multi_clip(plan, [hp], ranks.ws[r], scale=ranks.scale, skip=ranks.skip)
        zs.zs_mx4_quantize(ranks.full[0][:NUMELS[0]].view(torch.bfloat16).view(VOCAB, HIDDEN), b["wc"], b["ws"])
        zs.zs_mx4_quantize(x, b["xc"], b["xs"])
        zs.zs_mx4_matmul(b["xc"], b["xs"], b["wc"], b["ws"], b["y"])
        zs.zs_verify_drafts(b["y"], tokens, u, b["accepted"], b["out"], b["work"], logprobs=b["lps"])

    def inputs():
        x.normal_()
        tokens.random_(0, VOCAB)
        u.uniform_()
        for r in range(N):
            for q in range(N):
                for i, g in enumerate(pair[0].grads[r][q]):
                    g.copy_(torch.randn(g.shape, device="cuda").mul_(1e-2).bfloat16().view(torch.int16))
                    pair[1].grads[r][q][i].copy_(g)

    inputs()
    for ranks, b in zip(pair, bufs):
        calls(ranks, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(pair[0], bufs[0])
    for _ in range(3):
        inputs()
        graph.replay()
        calls(pair[1], bufs[1])
        torch.cuda.synchronize()
        for name in bufs[0]:
            if name != "work":
                assert torch.equal(bufs[0][name], bufs[1][name]), name
        for a, b in zip(pair[0].d, pair[1].d):
            for p, q in zip(a, b):
                assert all(torch.equal(p[name], q[name]) for name in p)
    for ranks in pair:
        ranks.close()
