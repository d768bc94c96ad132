"""The host code of the gated experts, the norms around a block and the
orthogonalised updates, built with AddressSanitizer and
UndefinedBehaviorSanitizer (g++, no GPU code) and driven by
tests/sanitize/gated_block_ortho_fuzz.cpp: random problems, strides and
addresses, with the launches checked instead of run."""
import os
import shutil
import subprocess

import pytest

from test_sanitizers import ENV, HERE, ROOT, SAN, _build


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_entry_points_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "dnn_conv2d_bwd_amd", "csrc")
    exe = _build(tmp_path, "gated_block_ortho_fuzz",
                 ["g++", "-std=c++17", *SAN, "-I", csrc, os.path.join(HERE, "gated_block_ortho_fuzz.cpp"),
                  *(os.path.join(csrc, f) for f in ("expert_api.cpp", "gated_api.cpp", "block_api.cpp", "ortho_api.cpp"))])
    r = subprocess.run([exe, "100000", "7"], capture_output=True, text=True, env=ENV, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr[-4000:]
    assert "launches:" in r.stdout
