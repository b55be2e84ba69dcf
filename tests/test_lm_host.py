"""Refusals and exports of the language-model operators that need no GPU: the
C calls reject every bad argument before they enqueue anything."""
import ctypes
import os
import re

import pytest

from conftest import import_zs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "zs_lm.h")


@pytest.fixture(scope="module")
def zs():
    return import_zs()


def test_exports_and_constants_match_the_header(zs):
    text = open(HEADER).read()
    declared = set(re.findall(r"^zs_status (zs_[a-z0-9_]+)\(", text, re.M))
    assert declared == set(zs.EXPORTED_LM) and len(declared) == 4
    raw = ctypes.CDLL(zs.LIB_PATH)
    assert all(hasattr(raw, s) for s in declared)
    macros = {m: int(v) for m, v in re.findall(r"#define\s+(ZS_[A-Z_]+)\s+(\d+)", text)}
    assert macros == {"ZS_QUANT_MATVEC_MAX_ROWS": zs.ZS_QUANT_MATVEC_MAX_ROWS,
                      "ZS_LOGPROBS_MAX_TOP": zs.ZS_LOGPROBS_MAX_TOP, "ZS_DISTILL_MAX_K": zs.ZS_DISTILL_MAX_K}
    assert re.search(r"ZS_DTYPE_BF16 = 0, ZS_DTYPE_F32 = 1", text)
    assert (zs.ZS_DTYPE_BF16, zs.ZS_DTYPE_F32) == (0, 1)


def _at(i):
    """A made-up device address far from every other one (never read: the calls fail first)."""
    return (i + 1) << 40


def _call(fn, good, **bad):
    args = dict(good, **bad)
    return fn(*args.values())


def _expect(zs, fn, good, status, **bad):
    assert _call(fn, good, **bad) == status, (bad, zs.zs_last_error())
    assert zs.zs_last_error()


def test_quant_matvec_refusals(zs):
    plan = zs.zs_shard_plan([64, 32 * 48], 2, 0, 64)
    per_tensor = zs.zs_shard_plan([32 * 48], 2, 0, layout=zs.ZS_LAYOUT_PER_TENSOR)
    good = dict(plan=plan.handle, tensor=1, out=32, n_in=48, bits=4, block=16, codes=_at(0), scales=_at(1), x=_at(2),
                x_stride=48, rows=3, y=_at(3), y_dtype=1, y_stride=32, stream=None)
    fn = zs.lib().zs_quant_matvec
    for bad in (dict(plan=None), dict(plan=per_tensor.handle, tensor=0), dict(tensor=-1), dict(tensor=2), dict(out=31),
                dict(out=-32, n_in=-48), dict(out=1 << 32, n_in=0), dict(bits=5), dict(block=24), dict(block=512),
                dict(rows=-1), dict(rows=65), dict(y_dtype=2), dict(x_stride=47), dict(y_stride=31),
                dict(x_stride=(1 << 40) + 1), dict(codes=None), dict(scales=None), dict(x=None), dict(y=None),
                dict(y=_at(2)), dict(y=_at(2) + 2 * (2 * 48 + 48) - 4), dict(y=_at(2) - 4 * (2 * 32 + 32) + 4),
                dict(y=_at(0)), dict(y=_at(1) + 4)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for bad in (dict(codes=_at(0) + 8), dict(scales=_at(1) + 4), dict(x=_at(2) + 1), dict(y=_at(3) + 2),
                dict(y=_at(3) + 1, y_dtype=0)):
        _expect(zs, fn, good, zs.ZS_EALIGN, **bad)
    assert _call(fn, good, rows=0, x=None, y=None) == zs.ZS_OK


LOGITS = dict(logits=_at(0), dtype=0, rows=4, vocab=100, stride=104)


def _logits_refusals(zs, fn, good):
    for bad in (dict(logits=None), dict(dtype=2), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 22), dict(vocab=0),
                dict(vocab=(1 << 30) + 1, stride=1 << 31), dict(stride=99), dict(stride=(1 << 40) + 1),
                dict(temperature=0.0), dict(temperature=-1.0), dict(temperature=float("nan")),
                dict(temperature=float("inf")), dict(temperature=1e-7)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    _expect(zs, fn, good, zs.ZS_EALIGN, logits=_at(0) + 1)
    _expect(zs, fn, good, zs.ZS_EALIGN, logits=_at(0) + 2, dtype=1)
    assert _call(fn, good, rows=0) == zs.ZS_OK


def test_strides_whose_extent_leaves_64_bits(zs):
    """(2^22 - 2) rows of fp32 2^40 elements apart end past 2^63 bytes."""
    _expect(zs, zs.lib().zs_token_logprobs,
            dict(LOGITS, dtype=1, tokens=_at(1), temperature=1.0, logprob=_at(2), entropy=None, stats=None, top=0,
                 ids=None, lps=None, stream=None), zs.ZS_EINVAL, rows=(1 << 22) - 1, stride=1 << 40)
    _expect(zs, zs.lib().zs_token_logprobs_backward,
            dict(LOGITS, dtype=1, tokens=_at(1), temperature=1.0, stats=_at(2), entropy=None, grad_logprob=_at(4),
                 grad_entropy=None, grad=_at(6), grad_stride=(1 << 38) + 1, stream=None), zs.ZS_EINVAL)


def test_token_logprobs_refusals(zs):
    good = dict(LOGITS, tokens=_at(1), temperature=1.0, logprob=_at(2), entropy=_at(3), stats=_at(4), top=2,
                ids=_at(5), lps=_at(6), stream=None)
    fn = zs.lib().zs_token_logprobs
    _logits_refusals(zs, fn, good)
    for bad in (dict(tokens=None), dict(top=-1), dict(top=33), dict(vocab=1, top=2), dict(ids=None), dict(lps=None),
                dict(top=0), dict(top=0, ids=None, lps=None, logprob=None, entropy=None, stats=None),
                dict(logprob=_at(3)), dict(stats=_at(2) + 4), dict(logprob=_at(0) + 4), dict(entropy=_at(1)),
                dict(lps=_at(5) + 4 * 7)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for name in ("tokens", "logprob", "entropy", "stats", "ids", "lps"):
        _expect(zs, fn, good, zs.ZS_EALIGN, **{name: good[name] + 2})


def test_token_logprobs_backward_refusals(zs):
    good = dict(LOGITS, tokens=_at(1), temperature=1.0, stats=_at(2), entropy=_at(3), grad_logprob=_at(4),
                grad_entropy=_at(5), grad=_at(6), grad_stride=100, stream=None)
    fn = zs.lib().zs_token_logprobs_backward
    _logits_refusals(zs, fn, good)
    for bad in (dict(tokens=None), dict(stats=None), dict(grad_logprob=None), dict(entropy=None), dict(grad=None),
                dict(grad_stride=99), dict(grad=_at(0)), dict(grad=_at(0) + 2, grad_stride=104),
                dict(grad=_at(0) + 2 * 104 * 3), dict(grad=_at(2)), dict(grad=_at(4) - 2 * 350)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for name in ("tokens", "stats", "entropy", "grad_logprob", "grad_entropy"):
        _expect(zs, fn, good, zs.ZS_EALIGN, **{name: good[name] + 2})
    _expect(zs, fn, good, zs.ZS_EALIGN, grad=_at(6) + 1)


def test_distill_refusals(zs):
    good = dict(LOGITS, ids=_at(1), teacher=_at(2), k=8, temperature=1.0, weight=_at(3), loss=_at(4), grad=_at(5),
                grad_stride=100, stream=None)
    fn = zs.lib().zs_distill_topk
    _logits_refusals(zs, fn, good)
    for bad in (dict(ids=None), dict(teacher=None), dict(loss=None), dict(k=0), dict(k=1025), dict(grad_stride=99),
                dict(grad=_at(0)), dict(loss=_at(0)), dict(loss=_at(1)), dict(loss=_at(5) + 8), dict(grad=_at(3))):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for name in ("ids", "teacher", "weight", "loss"):
        _expect(zs, fn, good, zs.ZS_EALIGN, **{name: good[name] + 2})


def test_binding_refuses_host_tensors(zs):
    import torch
    z, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_token_logprobs(z, t, logprob=torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_distill_topk(z, t[:, None], z[:, :1], torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_token_logprobs_backward(z, t, z[:, :2], z[:, 0], z)
    with pytest.raises(ValueError, match="CUDA"):
        zs.zs_quant_matvec(zs.zs_shard_plan([16], 1, 0), 0, 2, 8, 4, 8, None, None, z.bfloat16(), z)
