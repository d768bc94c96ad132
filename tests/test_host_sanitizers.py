"""The host code of the expert layer and of the gradient operators, built with
AddressSanitizer and UndefinedBehaviorSanitizer (g++, no GPU code) and driven by
tests/sanitize/expert_grad_fuzz.cpp: random problems, strides and addresses,
with the launches checked instead of run."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import ENV, HERE, ROOT, SAN, _build


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_entry_points_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "dnn_conv2d_bwd_amd", "csrc")
    exe = _build(tmp_path, "expert_grad_fuzz", ["g++", "-std=c++17", *SAN, "-I", csrc,
                                                os.path.join(HERE, "expert_grad_fuzz.cpp"),
                                                os.path.join(csrc, "expert_api.cpp"), os.path.join(csrc, "grad_api.cpp")])
    r = subprocess.run([exe, "100000", "7"], capture_output=True, text=True, env=ENV, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert "launches:" in r.stdout
