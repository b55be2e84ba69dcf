"""Host code of the language-model operators under the compiler's sanitizers (CPU only): argument validation at the
largest extents the calls accept, random arguments and concurrent callers (tests/sanitize/lm_driver.cpp)."""
import os
import shutil

import pytest

from test_sanitizers import ASAN_UBSAN, CSRC, ROOT, SAN, _build, _run

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")

SOURCES = [os.path.join(CSRC, f) for f in ("zs_api.cpp", "zs_lm_api.cpp", "zs_host_adamw.cpp")] + \
    [os.path.join(SAN, f) for f in ("host_stubs.cpp", "lm_driver.cpp")]


def _compile(tmp_path, flags):
    exe = str(tmp_path / "lm_san")
    _build(["g++", "-std=c++17", "-O1", "-g", "-ffp-contract=off", "-pthread", *flags, "-DZS_HOST_ONE_ISA",
            f"-I{os.path.join(ROOT, 'include')}", *SOURCES, "-o", exe])
    return exe


def test_host_calls_under_asan_ubsan(tmp_path):
    assert "lm driver ok (all)" in _run(_compile(tmp_path, ASAN_UBSAN), "all")


def test_host_calls_under_tsan(tmp_path):
    assert "lm driver ok (threads)" in _run(_compile(tmp_path, ["-fsanitize=thread"]), "threads")
