"""The rows that each lane of the norms' forward pass asks for, walked on the host
(CPU): a wave that takes several short rows at a time must not read a shared
gate's row for a row past the last, which would lie past the gate's end.  What
such a lane reads is dropped, so no result can show it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_implicit_gemm_conv2d_amd", "csrc")


def walk(csrc, folder):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    exe = str(folder / "row_walk")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", os.path.join(ROOT, "tests", "row_walk_host.cpp"), "-I", csrc,
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=60)


def test_no_lane_asks_for_a_row_that_does_not_exist(tmp_path):
    r = walk(CSRC, tmp_path)
    assert r.returncode == 0 and r.stdout.endswith(" walks\n"), r.stdout


def test_the_walk_finds_a_lane_that_asks_for_one(tmp_path):
    # the wave's end alone, without the lane's own row
    with open(os.path.join(CSRC, "row_walk.hpp")) as f:
        text = f.read()
    assert text.count("return sub < end - r;") == 1
    (tmp_path / "row_walk.hpp").write_text(text.replace("return sub < end - r;", "return r < end;"))
    assert walk(str(tmp_path), tmp_path).returncode == 1
