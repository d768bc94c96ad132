"""Which rows and tiles the workgroups of the expert products own: the code
that the kernels run (csrc/expert_device.h), built for the host with the lanes
of a wave emulated (tests/host/expert_tiles.cpp).  Every row of every feature
tile has exactly one workgroup, whatever the experts' sizes, also where the
last round's tiles are taken as halves."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_rows_and_tiles_are_owned_once(tmp_path):
    exe = os.path.join(str(tmp_path), "expert_tiles")
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-U_FORTIFY_SOURCE", "-I", os.path.join(ROOT, "dnn_conv2d_bwd_amd", "csrc"),
                        os.path.join(ROOT, "tests", "host", "expert_tiles.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe, "7", "24"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "cases: 24" in r.stdout
