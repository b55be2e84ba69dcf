"""Refusals and exports of the 4-bit format, the verification of drafted tokens and the clipped multi-tensor step that
need no GPU: the C calls reject every bad argument before they enqueue anything."""
import ctypes
import os
import re

import pytest

from conftest import import_zs

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def zs():
    return import_zs()


def test_exports_and_constants_match_the_headers(zs):
    raw = ctypes.CDLL(zs.LIB_PATH)
    macros = {}
    for header, names in (("zs_mx4.h", zs.EXPORTED_MX4), ("zs_drafts.h", zs.EXPORTED_DRAFTS),
                          ("zs_clip.h", zs.EXPORTED_CLIP)):
        text = open(os.path.join(ROOT, "include", header)).read()
        declared = re.findall(r"^(?:zs_status|int64_t) (zs_[a-z0-9_]+)\(", text, re.M)
        assert sorted(declared) == sorted(names) and all(hasattr(raw, s) for s in declared)
        macros.update((m, int(v)) for m, v in re.findall(r"#define\s+(ZS_[A-Z0-9_]+)\s+(\d+)", text))
    assert macros == {"ZS_MX4_BLOCK": zs.ZS_MX4_BLOCK, "ZS_VERIFY_MAX_DRAFTS": zs.ZS_VERIFY_MAX_DRAFTS}


@pytest.mark.parametrize("lang,std", [("c", "c11"), ("c++", "c++17")])
def test_headers_compile_alone(tmp_path, lang, std):
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    for header in ("zs_mx4.h", "zs_drafts.h", "zs_clip.h"):
        src = tmp_path / "h.c"
        src.write_text(f"#include <{header}>\nint main(void) {{ return 0; }}\n")
        subprocess.run(["gcc", "-x", lang, f"-std={std}", "-pedantic", "-Wall", "-Werror", "-fsyntax-only",
                        f"-I{os.path.join(ROOT, 'include')}", str(src)], check=True)


def _at(i):
    """A made-up device address far from every other one (never read: the calls fail first)."""
    return (i + 1) << 44


def _call(fn, good, **bad):
    return fn(*dict(good, **bad).values())


def _expect(zs, fn, good, status, **bad):
    assert _call(fn, good, **bad) == status, (bad, zs.zs_last_error())
    assert zs.zs_last_error()


QUANTIZE = dict(x=_at(0), dtype=0, rows=3, cols=70, stride=72, codes=_at(1), codes_stride=48, scales=_at(2),
                scales_stride=3, stream=None)
DEQUANTIZE = dict(codes=_at(1), codes_stride=48, scales=_at(2), scales_stride=3, rows=3, cols=70, x=_at(0), dtype=0,
                  stride=72, stream=None)


@pytest.mark.parametrize("name,good", [("zs_mx4_quantize", QUANTIZE), ("zs_mx4_dequantize", DEQUANTIZE)])
def test_conversion_refusals(zs, name, good):
    fn = getattr(zs.lib(), name)
    for bad in (dict(x=None), dict(codes=None), dict(scales=None), dict(dtype=2), dict(dtype=-1), dict(rows=-1),
                dict(rows=(1 << 25) + 1), dict(cols=-1), dict(cols=(1 << 34) + 1, stride=1 << 35), dict(stride=69),
                dict(stride=(1 << 38) + 1), dict(codes_stride=32), dict(scales_stride=2), dict(codes_stride=-48),
                dict(rows=1 << 25, stride=1 << 36), dict(x=_at(1)), dict(x=_at(1) + 48 * 2 + 46),
                dict(x=_at(1) - 2 * (72 * 2 + 70) + 2), dict(x=_at(2) - 2)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for bad in (dict(x=_at(0) + 1), dict(x=_at(0) + 2, dtype=1), dict(codes=_at(1) + 8), dict(codes_stride=56)):
        _expect(zs, fn, good, zs.ZS_EALIGN, **bad)
    assert _call(fn, good, rows=0, x=None) == zs.ZS_OK and _call(fn, good, cols=0, codes=None) == zs.ZS_OK
    if name == "zs_mx4_quantize":
        _expect(zs, fn, good, zs.ZS_EINVAL, scales=_at(1) + 47)


def test_matmul_refusals(zs):
    good = dict(xc=_at(0), xcs=64, xs=_at(1), xss=4, rows=5, wc=_at(2), wcs=80, ws=_at(3), wss=5, out=7, n_in=128,
                y=_at(4), dtype=1, stride=8, stream=None)
    fn = zs.lib().zs_mx4_matmul
    for bad in (dict(xc=None), dict(wc=None), dict(xs=None), dict(ws=None), dict(y=None), dict(rows=-1),
                dict(rows=(1 << 25) + 1), dict(out=-1), dict(out=(1 << 25) + 1), dict(n_in=-1),
                dict(n_in=(1 << 29) + 1, xcs=1 << 29, wcs=1 << 29, xss=1 << 29, wss=1 << 29), dict(dtype=2),
                dict(xcs=48), dict(wcs=48), dict(xss=3), dict(wss=3), dict(stride=6), dict(n_in=129),
                dict(y=_at(0)), dict(y=_at(1)), dict(y=_at(2) + 80 * 6 + 60), dict(y=_at(3) + 32),
                dict(y=_at(2) - 4 * (8 * 4 + 7) + 4)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for bad in (dict(xc=_at(0) + 4), dict(wc=_at(2) + 8), dict(xcs=72), dict(wcs=88), dict(y=_at(4) + 2),
                dict(y=_at(4) + 1, dtype=0)):
        _expect(zs, fn, good, zs.ZS_EALIGN, **bad)
    assert _call(fn, good, rows=0, xc=None, y=None) == zs.ZS_OK and _call(fn, good, out=0, wc=None) == zs.ZS_OK


def test_verify_refusals(zs):
    need = zs.zs_verify_drafts_workspace_bytes(3, 2, 100)
    good = dict(target=_at(0), dtype=0, requests=3, drafts=2, vocab=100, stride=104, draft=_at(1), dstride=100,
                tokens=_at(2), lens=_at(3), uniforms=_at(4), temperature=1.0, accepted=_at(5), out=_at(6),
                logprobs=_at(7), workspace=_at(8), bytes=need, stream=None)
    fn = zs.lib().zs_verify_drafts
    for bad in (dict(target=None), dict(tokens=None), dict(uniforms=None), dict(accepted=None), dict(out=None),
                dict(workspace=None), dict(dtype=2), dict(requests=-1), dict(requests=1 << 22), dict(drafts=-1),
                dict(drafts=65), dict(vocab=0), dict(vocab=(1 << 30) + 1, stride=1 << 31, dstride=1 << 31),
                dict(stride=99), dict(dstride=99), dict(stride=(1 << 38) + 1), dict(temperature=0.0),
                dict(temperature=float("nan")), dict(accepted=_at(6) + 32), dict(out=_at(0) + 4),
                dict(logprobs=_at(1) + 4), dict(accepted=_at(2) + 4), dict(out=_at(3) + 4), dict(logprobs=_at(4)),
                dict(workspace=_at(0)), dict(workspace=_at(7) + 32 - need // 16 * 16), dict(accepted=_at(8) + 4)):
        _expect(zs, fn, good, zs.ZS_EINVAL, **bad)
    for name in ("tokens", "lens", "uniforms", "accepted", "out", "logprobs", "workspace"):
        _expect(zs, fn, good, zs.ZS_EALIGN, **{name: good[name] + 2})
    _expect(zs, fn, good, zs.ZS_EALIGN, target=_at(0) + 1)
    _expect(zs, fn, good, zs.ZS_EALIGN, draft=_at(1) + 2, dtype=1)
    _expect(zs, fn, good, zs.ZS_ENOMEM, bytes=need - 1)
    assert _call(fn, good, requests=0, target=None) == zs.ZS_OK
    for bad in ((-1, 2, 100), (1 << 22, 0, 100), (3, 65, 100), (3, -1, 100), (3, 2, 0)):
        with pytest.raises(zs.ZsError):
            zs.zs_verify_drafts_workspace_bytes(*bad)
    assert zs.zs_verify_drafts_workspace_bytes(0, 0, 1) == 0


def test_clip_refusals(zs):
    L = zs.lib()
    plan = zs.zs_shard_plan([4096, 40], 4, 1, layout=zs.ZS_LAYOUT_PER_TENSOR)
    flat = zs.zs_shard_plan([4096, 40], 4, 1)
    assert L.zs_grad_stats_multi_workspace_bytes(None) == -1
    assert L.zs_grad_stats_multi_workspace_bytes(flat.handle) == -1
    need = L.zs_grad_stats_multi_workspace_bytes(plan.handle)
    assert need > 0
    hp = (zs.AdamWHParams * 1)(zs.AdamWHParams())
    for p in (None, flat.handle, plan.handle):  # no plan, no pieces, nothing bound
        assert L.zs_grad_stats_multi(p, _at(0), _at(1), _at(2), _at(3), need, None) == zs.ZS_EINVAL
        assert L.zs_adamw_shard_step_multi_clip(p, hp, 1, _at(1), _at(2), _at(0), None) == zs.ZS_EINVAL
    assert L.zs_grad_stats_multi(plan.handle, None, _at(1), _at(2), _at(3), need, None) == zs.ZS_EINVAL
