"""Calls at the edges of what the 4-bit format, the verification of drafted tokens and the multi-tensor norm allow:
random numbers from 1 on, rows and requests that are not to be read, calls at once on two streams."""
import math

import numpy as np
import pytest

from test_gpu_drafts import Case, zs  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests,k,vocab", [(40, 0, 5003), (40, 2, 1003), (1400, 2, 2051)])
def test_random_numbers_from_one_on_draw_the_last_token(zs, requests, k, vocab):
    """However the running sums round: the last token, or the last that exceeds its draft."""
    import torch
    c = Case(zs, requests, k, vocab, "f32", vocab)
    c.uniforms[:, k] = np.resize(np.array([1.0, 2.0, 3.0e38, math.inf], np.float32), requests)
    if k:
        c.uniforms[:, :k] = 2.0  # may stand where q is below p / 2
        c.draft.view(requests, k, vocab)[:, :, -1] = 60.0  # the last token is the draft's own
        c.target[:, -1] = 0.0
    c.device().call()
    torch.cuda.synchronize()
    at, out = c.out[0].cpu().numpy(), c.out[1].cpu().numpy()
    for b in range(requests):
        n = at[b]
        drawn = out[b, n]
        if n == k:
            assert drawn == vocab - 1
            continue
        p = torch.softmax(c.target.view(requests, k + 1, vocab)[b, n].double(), 0)
        q = torch.softmax(c.draft.view(requests, k, vocab)[b, n].double(), 0)
        over = torch.nonzero(p > q * (1 + 1e-12))
        assert drawn >= int(over[-1]) and drawn < vocab - 1 and float(p[drawn] - q[drawn]) > -1e-15


@pytest.mark.parametrize("requests,vocab", [(12, 1003), (600, 4099)])
def test_what_is_not_needed_is_not_read(zs, requests, vocab):
    """A padded batch: logits, tokens and random numbers behind a request's drafts, and all of a skipped request's, are
    NaN and out of range; the outputs are those of clean ones."""
    import torch
    k = 4
    lens = np.arange(requests) % (k + 2) - 1
    a, b = (Case(zs, requests, k, vocab, "f32", 5, lens=lens).device() for _ in range(2))
    for r in range(requests):
        n = int(lens[r])
        b.target.view(requests, k + 1, vocab)[r, n + 1 if n >= 0 else 0:] = math.nan
        b.draft.view(requests, k, vocab)[r, max(n, 0):] = math.nan
        b.d["tokens"][r, max(n, 0):] = -(1 << 31)
        b.d["uniforms"][r, max(n, 0):k] = math.nan
        if n < 0:
            b.d["uniforms"][r] = math.nan
    a.call()
    b.call()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a.out, b.out))
    assert not bool(torch.isnan(a.out[2]).any())


def test_calls_at_once_on_two_streams(zs):
    """Each with a workspace of its own; the results of calls alone."""
    import torch
    cases = [Case(zs, 30, 3, 20011, "f32", 1).device(), Case(zs, 7, 4, 32000, "bf16", 2).device()]
    streams = [torch.cuda.Stream() for _ in cases]
    x = [torch.randn(64, 2048, device="cuda") for _ in cases]
    w = [torch.randn(1000, 2048, device="cuda").bfloat16() for _ in cases]

    def u8(*shape):
        return torch.empty(*shape, dtype=torch.uint8, device="cuda")

    bufs = [dict(xc=u8(64, 1024), xs=u8(64, 64), wc=u8(1000, 1024), ws=u8(1000, 64),
                 y=torch.empty(64, 1000, device="cuda")) for _ in cases]

    def product(i, stream):
        b = bufs[i]
        zs.zs_mx4_quantize(x[i], b["xc"], b["xs"], stream=stream)
        zs.zs_mx4_quantize(w[i], b["wc"], b["ws"], stream=stream)
        zs.zs_mx4_matmul(b["xc"], b["xs"], b["wc"], b["ws"], b["y"], stream=stream)

    alone = []
    for i, c in enumerate(cases):
        c.call()
        product(i, None)
        torch.cuda.synchronize()
        alone.append([o.clone() for o in c.out] + [b.clone() for b in bufs[i].values()])
    for _ in range(5):
        for i, c in enumerate(cases):
            for t in list(c.out) + list(bufs[i].values()):
                t.fill_(3)
        torch.cuda.synchronize()
        for _ in range(3):
            for i, c in enumerate(cases):
                c.call(streams[i])
                product(i, streams[i])
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            assert all(torch.equal(p, q) for p, q in zip(alone[i], list(c.out) + list(bufs[i].values())))


def test_scalars_have_to_be_on_the_bindings_device(zs):
    import torch
    plan = zs.zs_shard_plan_ex([64, 8], 1, 0)
    d = [dict(grad=torch.zeros(n, dtype=torch.bfloat16, device="cuda"), master=torch.zeros(n, device="cuda"),
              m=torch.zeros(n, device="cuda"), v=torch.zeros(n, device="cuda")) for n in (64, 8)]
    ws = torch.zeros(zs.zs_multi_workspace_bytes(plan, 0), dtype=torch.uint8, device="cuda")
    zs.zs_multi_bind(plan, d, None, ws)
    good = dict(sumsq_out=torch.zeros(1, dtype=torch.float64, device="cuda"),
                nonfinite_out=torch.zeros(1, dtype=torch.int32, device="cuda"), workspace=ws,
                stats_workspace=torch.empty(zs.zs_grad_stats_multi_workspace_bytes(plan), dtype=torch.uint8,
                                            device="cuda"))
    for name in good:
        with pytest.raises(ValueError):
            zs.zs_grad_stats_multi(plan, **dict(good, **{name: good[name].cpu()}))
    with pytest.raises(ValueError):
        zs.zs_grad_stats_multi(plan, **dict(good, sumsq_out=good["sumsq_out"].float()))
    with pytest.raises(zs.ZsError):  # an output inside the bound table
        zs.zs_grad_stats_multi(plan, **dict(good, stats_workspace=ws))
    with pytest.raises(zs.ZsError):
        zs.zs_grad_stats_multi(plan, **dict(good, sumsq_out=ws[:8].view(torch.float64)))
    hp = zs.AdamWHParams(lr=1e-3, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1)
    for bad in (dict(scale=torch.ones(1)), dict(skip=torch.zeros(1, dtype=torch.int32)),
                dict(scale=torch.ones(1, dtype=torch.float64, device="cuda"))):
        with pytest.raises(ValueError):
            zs.zs_adamw_shard_step_multi_clip(plan, [hp], ws, **bad)
    zs.zs_grad_stats_multi(plan, **good)
    torch.cuda.synchronize()
    assert float(good["sumsq_out"]) == 0.0 and int(good["nonfinite_out"]) == 0
    zs.zs_multi_unbind(ws)
