"""Host code of the 4-bit format, the verification of drafted tokens and the clipped multi-tensor step under the
compiler's sanitizers (CPU only): argument validation at the largest extents the calls accept, random arguments, the
binding's tables and concurrent callers (tests/sanitize/more_driver.cpp)."""
import os
import shutil

import pytest

from test_sanitizers import ASAN_UBSAN, CSRC, ROOT, SAN, _build, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

SOURCES = [os.path.join(CSRC, f) for f in ("zs_api.cpp", "zs_mx4_api.cpp", "zs_drafts_api.cpp", "zs_clip_api.cpp",
                                           "zs_host_adamw.cpp")] + \
    [os.path.join(SAN, f) for f in ("host_stubs.cpp", "more_driver.cpp")]


def _compile(tmp_path, flags):
    exe = str(tmp_path / "more_san")
    _build(["g++", "-std=c++17", "-O1", "-g", "-ffp-contract=off", "-pthread", *flags, "-DZS_HOST_ONE_ISA",
            f"-I{os.path.join(ROOT, 'include')}", *SOURCES, "-o", exe])
    return exe


def test_host_calls_under_asan_ubsan(tmp_path):
    assert "more driver ok (all)" in _run(_compile(tmp_path, ASAN_UBSAN), "all")


def test_host_calls_under_tsan(tmp_path):
    assert "more driver ok (threads)" in _run(_compile(tmp_path, ["-fsanitize=thread"]), "threads")
