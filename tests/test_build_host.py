"""The build without a GPU: the C library needs neither torch nor its binding."""

import os
import subprocess
import sys

import pytest

from gradient_aggregation_gb300 import build
from tests.conftest import ROOT


def test_library_builds_where_torch_is_missing(fc_lib):
    """In a Python that cannot import torch, as for a user of the C ABI alone."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from gradient_aggregation_gb300 import build\n"
            "print(build.build_library())")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=600)
    assert out.returncode == 0, out.stderr
    assert out.stdout.strip() == build.LIB_PATH and os.path.exists(build.LIB_PATH)


def test_library_is_there_if_the_binding_cannot_be_built(fc_lib, monkeypatch, tmp_path):
    monkeypatch.setattr(build, "bind_path", lambda: str(tmp_path / "module.so"))
    monkeypatch.setattr(build, "_bind_command", lambda part: [sys.executable, "-c", "exit(1)"])
    assert build.build_library() == build.LIB_PATH
    with pytest.raises(RuntimeError, match="binding"):
        build.build_binding()
    with pytest.raises(RuntimeError, match="binding"):
        build.build_all()
    assert os.path.exists(build.LIB_PATH)


def test_binding_is_built_once(fc_lib):
    path = build.build_binding()
    stamp = os.path.getmtime(path)
    assert build.build_binding() == path and os.path.getmtime(path) == stamp
