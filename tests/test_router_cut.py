"""How the router's rows are cut into blocks, compiled for the host without CUDA: every shape
that the entry points accept, none at all among them, with undefined arithmetic trapped."""

import os
import shutil
import subprocess

import pytest

from gradient_aggregation_gb300 import build
from tests.conftest import ROOT


def test_rows_of_every_number_are_cut(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path / "router_cut")
    # traps need no library; aarch64 divides by zero without one
    p = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-fsanitize=undefined",
                        "-fsanitize-undefined-trap-on-error", "-I", build.CSRC,
                        os.path.join(ROOT, "tests", "c", "router_cut.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    p = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert p.returncode == 0, (p.returncode, p.stdout)
