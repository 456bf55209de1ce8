"""AdamW's tables on the host (CPU): the lists' elements once each, no launch past
the lanes that a grid holds, however large a list or a tensor is."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_implicit_gemm_conv2d_amd", "csrc")


def walk(csrc, folder):
    if shutil.which("g++") is None:
        pytest.skip("g++ is not available")
    exe = str(folder / "adamw_tables")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", os.path.join(ROOT, "tests", "adamw_tables_host.cpp"), "-I", csrc, "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([exe], capture_output=True, text=True, timeout=60)


def test_every_element_once_and_no_grid_too_large(tmp_path):
    r = walk(CSRC, tmp_path)
    assert r.returncode == 0 and r.stdout.endswith(" tables\n"), r.stdout


def test_the_walk_finds_a_table_without_an_end(tmp_path):
    with open(os.path.join(CSRC, "adamw_tables.hpp")) as f:
        text = f.read()
    assert text.count("left < room ? left : room") == 1
    (tmp_path / "adamw_tables.hpp").write_text(text.replace("left < room ? left : room", "left < room ? left : left"))
    assert walk(str(tmp_path), tmp_path).returncode == 1
