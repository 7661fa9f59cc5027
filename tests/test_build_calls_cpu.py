"""The compiled calls from torch (csrc/torch_calls.cpp) are optional: the library
is built without them, a module of another Python or torch is not taken, and one
that does not load leaves the way through ctypes."""
import os
import subprocess
import warnings

import pytest
import torch

from w8a8_gemm_b200 import binding as B
from w8a8_gemm_b200 import build as sqbuild


@pytest.fixture
def no_host_compiler(monkeypatch, tmp_path):
    """Compiled calls go to an empty folder, and no g++ command works."""
    run = subprocess.run

    def refuse(cmd, *a, **k):
        if os.path.basename(cmd[0]) == "g++":
            raise subprocess.CalledProcessError(1, cmd)
        return run(cmd, *a, **k)

    sqbuild.build()
    monkeypatch.setattr(sqbuild, "HERE", str(tmp_path))
    monkeypatch.setattr(sqbuild.subprocess, "run", refuse)


def test_the_library_is_built_without_them(no_host_compiler):
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert sqbuild.build() == sqbuild.LIB
    assert not os.path.exists(sqbuild.calls_path())


def test_a_module_of_an_older_source_does_not_stay(no_host_compiler):
    path = sqbuild.calls_path()
    with open(path, "wb"):
        pass
    os.utime(path, (0, 0))
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert sqbuild.build_calls() is None
    assert not os.path.exists(path)


def test_the_name_tells_python_and_torch(monkeypatch):
    here = sqbuild.calls_path()
    assert torch.__version__ in here
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    other = sqbuild.calls_path()
    assert other != here
    monkeypatch.undo()
    monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
    assert sqbuild.calls_path() not in (here, other)


@pytest.mark.parametrize("content", [None, b"not a module"])
def test_a_module_that_does_not_load_is_left_out(content, monkeypatch, tmp_path):
    sqbuild.build()
    path = tmp_path / "_sqtorch.other.so"
    if content is not None:
        path.write_bytes(content)
    monkeypatch.setattr(B, "calls_path", lambda: str(path))
    monkeypatch.setattr(B, "_native", None)
    with pytest.warns(RuntimeWarning, match="ctypes"):
        assert B._calls() is False
    with warnings.catch_warnings():          # said once
        warnings.simplefilter("error")
        assert B._calls() is False


def test_they_load_where_they_are_built(monkeypatch):
    sqbuild.build()
    path = sqbuild.build_calls()
    assert path and os.path.exists(path)
    monkeypatch.setattr(B, "_native", None)
    assert B._calls()
