"""Token log-probabilities, their gradient and top-logit distillation against
the 64-bit oracle (oracle/lm.py).

Tolerances, in units u = 2^-24 (half a step of fp32). An exponential e^d is off
by 4 u |d| (the difference, the factor log2(e) / T and their product round) and
4 u (the function). A sum of V of them is off by as many roundings as its
longest chain: below V / 256 + 64 however the kernels split rows over threads,
counting the rescalings to a new maximum; weighted with the distribution, |d|
is log V at most on average. So log s is off by
    tol_s = u (V / 256 + 68 + 4 log V),
log-probabilities by tol_s plus the roundings of d / T and of the result,
entropies by (2 + log V) tol_s twice over (a quotient of two such sums), and
probabilities by tol_s + 4 u |l| relatively. Every stored result is off by half
a step of its type on top.
"""
import math

import numpy as np
import pytest

from oracle import lm

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NAN, INF = math.nan, math.inf


@pytest.fixture(scope="module")
def zs():
    import torch

    import fsdp_sharded_mixed_flatten_amd as m
    torch.cuda.init()
    return m


def _dtype(name):
    import torch
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _half_step(name):
    return 2.0 ** -8 if name == "bf16" else U


def tol_s(vocab):
    return U * (vocab / 256 + 68 + 4 * math.log(vocab + 1))


def _logits(rows, vocab, dtype, seed=0, scale=3.0):
    import torch
    z = torch.randn(rows, vocab, generator=torch.Generator().manual_seed(seed)) * scale
    return z.to(_dtype(dtype))


def _near(got, want, tol, what):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape, what
    # a value of 2^128 - 2^103 or more rounds to infinity in fp32
    want = np.where(np.abs(want) >= 2.0 ** 128 - 2.0 ** 103, np.copysign(INF, want), want)
    special = ~np.isfinite(want)
    assert np.array_equal(got[special], want[special], equal_nan=True), what
    assert np.isfinite(got[~special]).all(), what
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want)
    bad = (off > np.broadcast_to(tol, want.shape)) & ~special
    assert not bad.any(), (what, int(bad.sum()), off[bad][:4], np.broadcast_to(tol, want.shape)[bad][:4])


class Forward:
    def __init__(self, rows, top):
        import torch
        full = lambda shape, v, dt=torch.float32: torch.full(shape, v, dtype=dt, device="cuda")  # noqa: E731
        self.out = {"logprob": full((rows,), -9.0), "entropy": full((rows,), -9.0), "stats": full((rows, 2), -9.0)}
        if top:
            self.out["top_ids"] = full((rows, top), -9, torch.int32)
            self.out["top_logprobs"] = full((rows, top), -9.0)

    def host(self):
        return {k: v.cpu().numpy().astype(np.float64) for k, v in self.out.items()}


def _check_forward(zs, z, tokens, temperature=1.0, top=0):
    """z: device logits (any view), tokens: list. Returns the forward outputs on the device."""
    import torch
    rows, vocab = z.shape
    f = Forward(rows, top)
    d_tokens = torch.tensor(tokens, dtype=torch.int32, device="cuda")
    zs.zs_token_logprobs(z, d_tokens, temperature=temperature, **f.out)
    ref = lm.token_logprobs(z.double().cpu().numpy(), tokens, temperature, top)
    got = f.host()
    ts = tol_s(vocab)
    lp_tol = lambda lp: ts + 6 * U * np.where(np.isfinite(lp), np.abs(lp), 0) + 4 * U * math.log(vocab + 1)  # noqa: E731
    _near(got["logprob"], ref["logprob"], lp_tol(ref["logprob"]), "logprob")
    _near(got["entropy"], ref["entropy"], 2 * (2 + math.log(vocab + 1)) * ts, "entropy")
    _near(got["stats"][:, 1], ref["stats"][:, 1], ts + 2 * U * math.log(vocab + 1), "log s")
    whole = ~np.isnan(ref["stats"][:, 0])
    assert np.array_equal(got["stats"][whole, 0], ref["stats"][whole, 0]), "max"
    if top:
        assert np.array_equal(got["top_ids"], ref["top_ids"]), "top_ids"
        _near(got["top_logprobs"], ref["top_logprobs"], lp_tol(ref["top_logprobs"]), "top_logprobs")
    return f, d_tokens


VOCABS = [1, 2, 7, 8, 9, 63, 64, 257, 1000, 2048, 2049, 4100, 8191, 8192, 16385, 32000, 32768, 50007, 65543]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprobs(zs, vocab, dtype):
    rng = np.random.default_rng(vocab)
    for temperature, top in ((1.0, min(vocab, 20)), (0.6, min(vocab, 1)), (1.7, 0), (1.0, min(vocab, 32))):
        z = _logits(5, vocab, dtype, seed=vocab + top).cuda()
        tokens = rng.integers(0, vocab, 5).tolist()
        tokens[3] = -1
        _check_forward(zs, z, tokens, temperature, top)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 128256), ("f32", 151936), ("bf16", 163841), ("f32", 200003)])
def test_logprobs_large_vocabularies(zs, vocab, dtype):
    z = _logits(3, vocab, dtype, seed=1).cuda()
    _check_forward(zs, z, [5, vocab - 1, vocab // 2], 0.9, 32)


def _special_rows(vocab):
    """(name, logits row, token): masks and ties as they come."""
    rng = np.random.default_rng(7)
    base = rng.standard_normal(vocab) * 2
    rows = []
    few = np.full(vocab, -INF)
    few[[vocab // 3, vocab // 2, vocab - 1]] = [1.0, 2.0, 2.0]
    rows.append(("three allowed", few, vocab // 2))
    rows.append(("token masked", few, 0))
    rows.append(("one allowed", np.where(np.arange(vocab) == vocab - 2, 5.0, -INF), vocab - 2))
    rows.append(("none allowed", np.full(vocab, -INF), 1))
    rows.append(("all equal", np.zeros(vocab), 3))
    rows.append(("all lowest", np.full(vocab, -3.38e38), 3))
    rows.append(("lowest beside others", np.where(np.arange(vocab) % 3 == 0, base, -3.38e38), 3))
    rows.append(("lowest and masked", np.where(np.arange(vocab) % 3 == 0, -3.38e38, -INF), 3))
    rows.append(("signed zeros", np.where(np.arange(vocab) % 2 == 0, -0.0, 0.0), 1))
    rows.append(("rising", np.linspace(-50, 50, vocab), vocab - 1))
    rows.append(("falling", np.linspace(50, -50, vocab), 0))
    rows.append(("few values", rng.integers(0, 3, vocab).astype(float), 2))
    rows.append(("far apart", np.where(np.arange(vocab) == 5, 3e38, base), 5))
    nan, inf = base.copy(), base.copy()
    nan[vocab // 2] = NAN
    inf[vocab // 2] = INF
    rows.append(("a NaN", nan, 0))
    rows.append(("an infinity", inf, vocab // 2))
    rows.append(("token past the end", base, vocab))
    rows.append(("token far past the end", base, 2 ** 31 - 1))
    rows.append(("skipped", nan, -100))
    return rows


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 3000, 40001, 110003])
def test_logprobs_masks_ties_and_specials(zs, vocab, dtype):
    import torch
    rows = _special_rows(vocab)
    z = torch.tensor(np.array([r[1] for r in rows])).to(_dtype(dtype)).cuda()
    for top in (0, 1, 20):
        _check_forward(zs, z, [r[2] for r in rows], 1.0, top)
    _check_forward(zs, z, [r[2] for r in rows], 0.5, 8)


def test_optional_outputs(zs):
    import torch
    z = _logits(3, 100, "f32").cuda()
    tokens = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    whole = Forward(3, 4)
    zs.zs_token_logprobs(z, tokens, **whole.out)
    for names in (("logprob",), ("entropy",), ("stats",), ("top_ids", "top_logprobs")):
        f = Forward(3, 4)
        zs.zs_token_logprobs(z, tokens, **{n: f.out[n] for n in names})
        for n, v in f.out.items():
            assert torch.equal(v, whole.out[n]) if n in names else (v == -9).all()


# ---------------------------------------------------------------- gradient of the log-probabilities


def _grad_tol(ref, mag, vocab, dtype, z, temperature, factor):
    """mag: the terms' magnitude before they cancel. factor: what a probability is multiplied with at most, a number a
    row: an exponential below 2^-126 counts as 0, which takes up to 2^-126 from a probability (exponentials are
    divided by a sum that is at least about 1) and so up to 2^-126 factor from the gradient."""
    with np.errstate(invalid="ignore"):
        spread = np.nanmax(np.where(np.isfinite(z), z, -INF), axis=1, keepdims=True) - z
        l = np.where(np.isfinite(spread), np.minimum(spread / temperature, 110.0), 0) + math.log(vocab + 1)
    return mag * (2 * tol_s(vocab) + 16 * U + 8 * U * l) + _half_step(dtype) * np.abs(ref) * (1 + 1e-3) \
        + 2.0 ** -126 * (1 + np.asarray(factor)[:, None])


def _check_gradient(zs, z, tokens, temperature, with_entropy, grad=None):
    import torch
    rows, vocab = z.shape
    dtype = "bf16" if z.dtype == torch.bfloat16 else "f32"
    host = z.double().cpu().numpy()
    f, d_tokens = _check_forward(zs, z, tokens, temperature)
    rng = np.random.default_rng(rows)
    gl = torch.tensor(rng.standard_normal(rows), dtype=torch.float32, device="cuda")
    gh = torch.tensor(rng.standard_normal(rows), dtype=torch.float32, device="cuda") if with_entropy else None
    g = torch.full((rows, vocab), 7.0, dtype=z.dtype, device="cuda") if grad is None else grad
    zs.zs_token_logprobs_backward(z, d_tokens, f.out["stats"], gl, g, temperature=temperature,
                                  entropy=f.out["entropy"] if with_entropy else None, grad_entropy=gh)
    ref, mag = lm.token_logprobs_backward(host, tokens, temperature, gl.cpu().numpy(),
                                          gh.cpu().numpy() if with_entropy else None)
    # the entropy that the gradient takes is itself off by its own tolerance
    if with_entropy:
        mag = mag + np.abs(gh.cpu().numpy())[:, None] * 2 * (2 + math.log(vocab + 1)) / temperature * np.exp(
            np.array([lm.row_softmax(r, temperature)[2] for r in host]))
    # |l| where p is not 0 yet: below log 2^150
    factor = np.abs(gl.cpu().numpy()) / temperature
    if with_entropy:
        factor = factor + np.abs(gh.cpu().numpy()) * (104 + math.log(vocab + 1)) / temperature
    _near(g.double().cpu().numpy(), ref, _grad_tol(ref, mag, vocab, dtype, host, temperature, factor), "grad_logits")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_logprobs_gradient(zs, vocab, dtype):
    rng = np.random.default_rng(vocab)
    tokens = rng.integers(0, vocab, 4).tolist() + [-1]
    for temperature, with_entropy in ((1.0, True), (0.7, False), (1.6, True)):
        _check_gradient(zs, _logits(5, vocab, dtype, seed=vocab).cuda(), tokens, temperature, with_entropy)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_gradient_specials(zs, dtype):
    import torch
    vocab = 3001
    rows = _special_rows(vocab)
    z = torch.tensor(np.array([r[1] for r in rows])).to(_dtype(dtype)).cuda()
    # a masked token's log-probability has no gradient that means anything to the loss, but it has the formula's
    for with_entropy in (False, True):
        _check_gradient(zs, z, [r[2] for r in rows], 1.0, with_entropy)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [1, 9, 3001, 40001])
def test_nan_among_masked_logits(zs, vocab, dtype):
    """A NaN is not hidden by the row's maximum being -infinity."""
    import torch
    z = torch.full((3, vocab), -INF, dtype=_dtype(dtype), device="cuda")
    z[0, 0] = z[1, vocab - 1] = z[2, vocab // 2] = NAN
    tokens = [vocab - 1, 0, vocab // 3]
    _check_forward(zs, z, tokens, 1.0, min(vocab, 4))
    for with_entropy in (False, True):
        _check_gradient(zs, z, tokens, 1.0, with_entropy)


def test_gradient_equals_differences(zs):
    """The gradient against central differences of the forward call itself (fp32 logits, a step of 2^-5: truncation
    h^2 / 6 times a third derivative below 2 g, rounding 2 tol / 2h)."""
    import torch
    vocab, h = 64, 2.0 ** -5
    z = _logits(1, vocab, "f32", seed=3, scale=1.5)
    tokens = torch.full((vocab,), 9, dtype=torch.int32, device="cuda")
    gl, gh = 0.7, -0.4

    def value(x):
        lp, en = torch.empty(vocab, device="cuda"), torch.empty(vocab, device="cuda")
        zs.zs_token_logprobs(x, tokens, logprob=lp, entropy=en)
        return gl * lp.double() + gh * en.double()

    eye = torch.eye(vocab) * h
    diff = (value((z + eye).cuda()) - value((z - eye).cuda())) / (2 * h)
    zc = z.cuda()
    f, _ = _check_forward(zs, zc, [9])
    g = torch.empty_like(zc)
    zs.zs_token_logprobs_backward(zc, tokens[:1], f.out["stats"], torch.tensor([gl], device="cuda"), g,
                                  entropy=f.out["entropy"], grad_entropy=torch.tensor([gh], device="cuda"))
    # third derivatives of logprob and entropy along one logit: at most 1 and 1 + 4 log V
    third = abs(gl) + abs(gh) * (1 + 4 * math.log(vocab))
    tol = h * h / 6 * third + 2 * (2 + math.log(vocab)) * tol_s(vocab) * 2 / h
    assert (diff - g[0].double()).abs().max().item() <= tol


# ---------------------------------------------------------------- distillation


def _check_distill(zs, z, ids, teacher, temperature=1.0, weight=None, grad=None):
    import torch
    rows, vocab = z.shape
    dtype = "bf16" if z.dtype == torch.bfloat16 else "f32"
    host = z.double().cpu().numpy()
    d_ids = torch.tensor(np.asarray(ids), dtype=torch.int32, device="cuda")
    d_teacher = torch.tensor(np.asarray(teacher), dtype=torch.float32, device="cuda")
    d_w = None if weight is None else torch.tensor(weight, dtype=torch.float32, device="cuda")
    k = d_ids.shape[1]
    ref, lmag, g_ref, g_mag = lm.distill_topk(host, np.asarray(ids), d_teacher.double().cpu().numpy(), temperature,
                                              None if weight is None else d_w.double().cpu().numpy())
    t_top = np.where(np.asarray(ids) >= 0, d_teacher.cpu().numpy(), -INF)
    with np.errstate(invalid="ignore"):
        reach = np.nanmax(np.where(np.isfinite(t_top), t_top, -INF), axis=1) - np.nanmin(
            np.where(np.isfinite(t_top), t_top, INF), axis=1)
    reach = np.where(np.isfinite(reach), np.minimum(reach / temperature, 110.0), 0)
    # the teacher's q: k exponentials of differences up to `reach` and their sum
    tol_q = U * (k + 16 + 8 * reach)
    scale = np.ones(rows) if weight is None else np.abs(np.asarray(weight, float))
    scale = np.where(np.isfinite(scale), scale, 0)
    loss = torch.full((rows,), -9.0, device="cuda")
    zs.zs_distill_topk(z, d_ids, d_teacher, loss, temperature=temperature, row_weight=d_w)
    tol = (lmag + scale * temperature ** 2 * math.log(vocab + 1)) * (2 * tol_q + 16 * U) \
        + 2 * scale * temperature ** 2 * tol_s(vocab)
    _near(loss.cpu().numpy(), ref, tol, "loss")
    alone = loss.clone()
    loss.fill_(-9.0)
    g = torch.full((rows, vocab), 7.0, dtype=z.dtype, device="cuda") if grad is None else grad
    zs.zs_distill_topk(z, d_ids, d_teacher, loss, grad_logits=g, temperature=temperature, row_weight=d_w)
    assert torch.equal(alone.view(torch.int32), loss.view(torch.int32))
    g_tol = _grad_tol(g_ref, g_mag, vocab, dtype, host, temperature, scale * temperature) + g_mag * tol_q[:, None]
    _near(g.double().cpu().numpy(), g_ref, g_tol, "grad_logits")


def _teacher(rng, rows, k, vocab):
    ids = np.array([rng.permutation(vocab)[:k] if k <= vocab else rng.integers(0, vocab, k) for _ in range(rows)])
    return ids, rng.standard_normal((rows, k)) * 3


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_distill(zs, vocab, dtype):
    rng = np.random.default_rng(vocab)
    for k, temperature, weighted in ((1, 1.0, False), (7, 2.0, True), (64, 0.7, True), (300, 1.0, False)):
        ids, teacher = _teacher(rng, 4, k, vocab)
        ids[1, k // 2:] = -1  # ragged; all of the row's entries unused where k is 1
        z = _logits(4, vocab, dtype, seed=vocab + k)
        _check_distill(zs, z.cuda(), ids, teacher, temperature, [0.25, 1.0, 0.0, 2.5] if weighted else None)


@pytest.mark.parametrize("dtype,vocab,k", [("bf16", 128256, 64), ("f32", 151936, 1024), ("bf16", 163841, 128),
                                           ("f32", 81921, 5), ("bf16", 163840, 1), ("bf16", 131072, 2),
                                           ("f32", 65536, 33), ("f32", 81920, 3)])
def test_distill_large_vocabularies(zs, vocab, dtype, k):
    rng = np.random.default_rng(k)
    ids, teacher = _teacher(rng, 2, k, vocab)
    ids[0, 0] = vocab - 1
    ids[1, 0] = 0
    _check_distill(zs, _logits(2, vocab, dtype, seed=2).cuda(), ids, teacher, 2.0, [1.0, 0.5])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab", [40, 3000, 70003])
def test_distill_specials(zs, vocab, dtype):
    import torch
    special = [r for r in _special_rows(vocab)]
    rows = len(special)
    rng = np.random.default_rng(5)
    ids, teacher = _teacher(rng, rows, 12, vocab)
    z = torch.tensor(np.array([r[1] for r in special])).to(_dtype(dtype))
    _check_distill(zs, z.cuda(), ids, teacher, 1.0)
    # the teacher's side: an id twice (three times), masked entries, none left, a NaN, an infinity, an id past the end,
    # a skipped row over NaN logits, a NaN in an unused entry
    z = _logits(10, vocab, dtype, seed=1)
    ids, teacher = _teacher(rng, 10, 12, vocab)
    ids[0, 3] = ids[0, 7] = ids[0, 11] = ids[0, 0]
    ids[0, 5] = ids[0, 4]
    teacher[1, ::2] = -INF
    teacher[2] = -INF
    ids[3] = -1
    teacher[4, 2] = NAN
    teacher[5, 2] = INF
    ids[6, 1] = vocab
    z[7, 3] = NAN
    teacher[8, 6] = NAN
    ids[8, 6] = -5
    ids[9, 6] = 2 ** 31 - 1
    weight = [1.0, 0.5, 1.0, 1.0, 1.0, 1.0, 1.0, 0.0, 2.0, 0.0]
    _check_distill(zs, z.cuda(), ids, teacher, 1.5, weight)
    # a token masked in the student that the teacher wants: an infinite loss, a finite gradient
    z = _logits(2, vocab, dtype, seed=4)
    z[0, int(ids[0, 1])] = -INF
    _check_distill(zs, z.cuda(), ids[:2], teacher[:2])


# ---------------------------------------------------------------- memory, streams, graphs


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("vocab,pad,shift", [(1000, 24, 0), (1001, 0, 1), (4099, 2, 3), (33000, 5, 1)])
def test_strided_rows_and_guards(zs, vocab, pad, shift, dtype):
    """Logits and gradients as views whose rows start anywhere; what lies between rows is neither read nor written."""
    import torch
    rows = 4
    big = torch.full((rows + 2, vocab + pad + shift), NAN, dtype=_dtype(dtype))
    big[1:1 + rows, shift:shift + vocab] = _logits(rows, vocab, dtype, seed=8)
    d = big.cuda()
    z = d[1:1 + rows, shift:shift + vocab]
    tokens = [0, vocab - 1, 5, -1]
    rng = np.random.default_rng(0)
    ids, teacher = _teacher(rng, rows, 9, vocab)
    _check_forward(zs, z, tokens, 1.0, 5)

    def guards_hold(buf, off):
        b = buf.clone()
        b[1:1 + rows, off:off + vocab] = 3.0
        return bool((b == 3.0).all())

    for off in (0, 2, 7):
        buf = torch.full((rows + 2, vocab + 11), 3.0, dtype=_dtype(dtype), device="cuda")
        _check_gradient(zs, z, tokens, 1.0, True, grad=buf[1:1 + rows, off:off + vocab])
        assert guards_hold(buf, off)
        buf.fill_(3.0)
        _check_distill(zs, z, ids, teacher, 1.0, None, grad=buf[1:1 + rows, off:off + vocab])
        assert guards_hold(buf, off)


@pytest.mark.parametrize("dtype,vocab", [("bf16", 5003), ("f32", 32000), ("bf16", 131080), ("f32", 90001),
                                         ("bf16", 170001)])
def test_in_place_gradients(zs, vocab, dtype):
    """grad_logits = logits gives the bits of the separate call."""
    import torch
    z = _logits(3, vocab, dtype, seed=6).cuda()
    tokens = torch.tensor([1, -1, vocab - 1], dtype=torch.int32, device="cuda")
    f = Forward(3, 0)
    zs.zs_token_logprobs(z, tokens, **f.out)
    gl, gh = torch.tensor([1.0, 2.0, -3.0], device="cuda"), torch.tensor([0.1, 0.2, -0.3], device="cuda")
    kw = dict(entropy=f.out["entropy"], grad_entropy=gh)
    apart, own = torch.empty_like(z), z.clone()
    zs.zs_token_logprobs_backward(z, tokens, f.out["stats"], gl, apart, **kw)
    zs.zs_token_logprobs_backward(own, tokens, f.out["stats"], gl, own, **kw)
    assert torch.equal(apart, own)
    rng = np.random.default_rng(1)
    ids, teacher = _teacher(rng, 3, 40, vocab)
    ids[2, 3] = ids[2, 4]
    d_ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
    d_te = torch.tensor(teacher, dtype=torch.float32, device="cuda")
    loss, loss2, own = torch.empty(3, device="cuda"), torch.empty(3, device="cuda"), z.clone()
    zs.zs_distill_topk(z, d_ids, d_te, loss, grad_logits=apart)
    zs.zs_distill_topk(own, d_ids, d_te, loss2, grad_logits=own)
    assert torch.equal(apart, own) and torch.equal(loss, loss2)


def test_many_rows_and_repeats(zs):
    """More rows than the chip holds blocks; the same bits every time."""
    import torch
    rows, vocab = 3001, 1030
    z = _logits(rows, vocab, "bf16", seed=2).cuda()
    tokens = (torch.arange(rows, device="cuda") * 7 % (vocab + 30) - 30).to(torch.int32)
    f, _ = _check_forward(zs, z, tokens.cpu().tolist(), 1.0, 3)
    again = Forward(rows, 3)
    zs.zs_token_logprobs(z, tokens, **again.out)
    assert all(torch.equal(f.out[n], again.out[n]) for n in f.out)
    gl = torch.linspace(-1, 1, rows, device="cuda")
    g = [torch.empty_like(z) for _ in range(2)]
    for x in g:
        zs.zs_token_logprobs_backward(z, tokens, f.out["stats"], gl, x)
    assert torch.equal(g[0], g[1])


def test_rows_past_32_bit_offsets(zs):
    """Rows behind 2^31 elements (4 GiB) of logits: first and last rows of a long batch."""
    import torch
    vocab = 1 << 19
    rows = (1 << 31) // vocab + 2
    z = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    part = _logits(2, vocab, "bf16", seed=3)
    z[-2:] = part.cuda()
    tokens = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    tokens[-2:] = torch.tensor([3, vocab - 1], dtype=torch.int32, device="cuda")
    f = Forward(rows, 2)
    zs.zs_token_logprobs(z, tokens, **f.out)
    small, _ = _check_forward(zs, part.cuda(), [3, vocab - 1], 1.0, 2)
    for n in f.out:
        assert torch.equal(f.out[n][-2:], small.out[n])
    gl = torch.ones(rows, device="cuda")
    g_small = torch.empty_like(part, device="cuda")
    zs.zs_token_logprobs_backward(part.cuda(), tokens[-2:].clone(), small.out["stats"], gl[:2], g_small)
    zs.zs_token_logprobs_backward(z, tokens, f.out["stats"], gl, z)  # in place
    assert torch.equal(z[-2:], g_small) and not z[:-2].any()


def test_gradient_of_more_work_than_a_launch(zs):
    """2^22 - 1 rows of 5 workgroups each, in place: more work-items than 2^32. All but a few rows are skipped."""
    import torch
    rows, vocab = (1 << 22) - 1, 16392
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 138 GB of device memory")
    z = torch.empty(rows, vocab, dtype=torch.bfloat16, device="cuda")
    split = ((1 << 32) - 1) // 256 // 5  # rows of the first launch
    live = torch.tensor([0, split - 1, split, rows - 1], device="cuda")
    part = _logits(4, vocab, "bf16", seed=4).cuda()
    z[live] = part
    z[split + 1] = 5.0  # a skipped row that has to become 0
    tokens = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
    tokens[live] = torch.tensor([0, 5, 16391, 77], dtype=torch.int32, device="cuda")
    f, _ = _check_forward(zs, part, [0, 5, 16391, 77])
    stats = torch.zeros(rows, 2, device="cuda")
    stats[live] = f.out["stats"]
    gl = torch.linspace(0.5, 1.5, rows, device="cuda")
    want = torch.empty_like(part)
    zs.zs_token_logprobs_backward(part, tokens[live], f.out["stats"], gl[live], want)
    zs.zs_token_logprobs_backward(z, tokens, stats, gl, z)
    assert torch.equal(z[live], want)
    for r in (1, split - 2, split + 1, rows - 2):
        assert not z[r].any()
    del z
    torch.cuda.empty_cache()


def test_streams_and_graph(zs):
    """A forward call and its gradient captured together, replayed on new inputs with eager work between, on a side
    stream, and two at once."""
    import torch
    rows, vocab = 6, 5000
    zs_in = [_logits(rows, vocab, "bf16", seed=s).cuda() for s in range(4)]
    tokens = torch.tensor([1, 2, -1, 4, 5, 4999], dtype=torch.int32, device="cuda")
    gl = torch.linspace(0.5, 1.5, rows, device="cuda")
    rng = np.random.default_rng(0)
    ids, teacher = _teacher(rng, rows, 16, vocab)
    d_ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
    d_te = torch.tensor(teacher, dtype=torch.float32, device="cuda")

    class Run:
        def __init__(self):
            self.f, self.g, self.dg = Forward(rows, 4), torch.empty_like(zs_in[0]), torch.empty_like(zs_in[0])
            self.loss = torch.empty(rows, device="cuda")

        def go(self, z, **kw):
            zs.zs_token_logprobs(z, tokens, **self.f.out, **kw)
            zs.zs_token_logprobs_backward(z, tokens, self.f.out["stats"], gl, self.g, entropy=self.f.out["entropy"],
                                          grad_entropy=gl, **kw)
            zs.zs_distill_topk(z, d_ids, d_te, self.loss, grad_logits=self.dg, **kw)

        def all(self):
            return list(self.f.out.values()) + [self.g, self.dg, self.loss]

    want = []
    for z in zs_in:
        r = Run()
        r.go(z)
        want.append(r)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    runs = [Run() for _ in zs_in]
    torch.cuda.synchronize()
    for i, z in enumerate(zs_in):
        runs[i].go(z, stream=streams[i % 2])
    torch.cuda.synchronize()
    for a, b in zip(runs, want):
        assert all(torch.equal(x, y) for x, y in zip(a.all(), b.all()))
    static, r = zs_in[0].clone(), Run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r.go(static)
    eager = Run()
    for i in (2, 0, 3, 1):
        static.copy_(zs_in[i])
        graph.replay()
        eager.go(zs_in[(i + 1) % 4])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(r.all(), want[i].all()))
        assert all(torch.equal(x, y) for x, y in zip(eager.all(), want[(i + 1) % 4].all()))


def test_binding_refusals(zs):
    import torch
    z = _logits(3, 50, "bf16").cuda()
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    f = torch.zeros(3, device="cuda")
    ids = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    te = torch.zeros(3, 4, device="cuda")
    bad_forward = [dict(tokens=t.long()), dict(tokens=t[:2]), dict(tokens=t.cpu()), dict(logits=z.half()),
                   dict(logits=z.t().contiguous().t()), dict(logits=z[0]), dict(logprob=f.double()),
                   dict(top_ids=ids), dict(top_logprobs=te), dict(top_ids=ids[:2], top_logprobs=te)]
    for bad in bad_forward:
        with pytest.raises(ValueError):
            zs.zs_token_logprobs(**{**dict(logits=z, tokens=t, logprob=f), **bad})
    for bad in (dict(grad_logits=z.float()), dict(grad_logits=z[:2]), dict(stats=f), dict(grad_logprob=f[:1])):
        with pytest.raises(ValueError):
            zs.zs_token_logprobs_backward(**{**dict(logits=z, tokens=t, stats=torch.zeros(3, 2, device="cuda"),
                                                    grad_logprob=f, grad_logits=torch.empty_like(z)), **bad})
    for bad in (dict(teacher_ids=ids[:, :3]), dict(teacher_logits=te.bfloat16()), dict(loss=f[:2]),
                dict(row_weight=te), dict(grad_logits=z.float())):
        with pytest.raises(ValueError):
            zs.zs_distill_topk(**{**dict(logits=z, teacher_ids=ids, teacher_logits=te, loss=f), **bad})
    with pytest.raises(zs.ZsError):
        zs.zs_token_logprobs(z, t)
    with pytest.raises(zs.ZsError):
        zs.zs_token_logprobs(z, t, logprob=f, temperature=0.0)
    with pytest.raises(zs.ZsError):  # overlapping, and not the logits themselves
        zs.zs_token_logprobs_backward(z[:2], t[:2], torch.zeros(2, 2, device="cuda"), f[:2], z[1:])
