"""Shared-memory layouts of the loss kernels, checked where the compiler knows them: the kernels' source is compiled
for the host (syntax only, nothing runs) with assertions on the sizes that its reductions rely on."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fsdp_sharded_mixed_flatten_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None, reason="needs hipcc")


def _compiles(tmp_path, asserted):
    src = tmp_path / "layout.hip"
    src.write_text('#include "zs_loss.hip"\n' + "".join(f"static_assert({a}, \"\");\n" for a in asserted))
    return subprocess.run(["hipcc", "--offload-arch=gfx950", "-std=c++17", "-fsyntax-only", "--cuda-host-only",
                           f"-I{CSRC}", f"-I{os.path.join(ROOT, 'include')}", str(src)], capture_output=True, text=True)


def test_the_check_itself_fails_on_a_false_size(tmp_path):
    assert _compiles(tmp_path, []).returncode == 0
    assert _compiles(tmp_path, ["sizeof(zs::Fast) == 1"]).returncode != 0


def test_distillation_holds_the_sums_of_every_wave(tmp_path):
    """A workgroup of 1024 threads has 16 waves, each of which leaves its sums (of either form) in `part`."""
    part = "sizeof(zs::DistillShared::part)"
    res = _compiles(tmp_path, [f"{part} >= 16 * sizeof(zs::{form})" for form in ("Running", "Fast")])
    assert res.returncode == 0, res.stderr[-2000:]
