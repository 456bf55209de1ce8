"""A launch of 2^32 lanes or more in a dimension (CPU): the runtime leaves lanes out
without a word, so it is refused on the host."""
import os
import subprocess

import pytest

from convolution_implicit_gemm_conv2d_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_launches_that_no_grid_holds_are_refused(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("hipcc is not available")
    exe = str(tmp_path / "launch")
    r = subprocess.run([build.HIPCC, *build.CFLAGS, os.path.join(ROOT, "tests", "launch_host.hip"), "-I", build.CSRC, "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "4 refused\n", r.stdout
