"""Host check of the rules that attention over shared prefixes divides its work by.

Compiles tests/branch_cost_check.cpp (g++) against the library's branch_cost.h,
the code that the kernels and their launches use, and runs it."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_tiles_count_for_what_they_take(tmp_path):
    exe = tmp_path / "branch_cost_check"
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", os.path.join(ROOT, "tests", "branch_cost_check.cpp"),
                    "-o", str(exe)], check=True, capture_output=True, text=True)
    res = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.strip().startswith("ok")
