"""The MXFP4 product's rules that are plain arithmetic, compiled for the host (no GPU)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "sigmoid_top_routing_02_amd", "csrc")

pytestmark = pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not found")


def _run(name, tmp_path):
    exe = str(tmp_path / name)
    r = subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-I", CSRC, "-o", exe,
                        os.path.join(ROOT, "tests", "host", name + ".cpp")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    return r.stdout


def test_offsets_stay_inside_the_tensors(tmp_path):
    assert "reads checked" in _run("mx_offsets", tmp_path)


def test_few_row_launches_stay_under_their_limits(tmp_path):
    assert "few rows" in _run("mx_choose", tmp_path)
