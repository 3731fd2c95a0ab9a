"""The library's build where the binding's extension cannot be built: libfno.so is a plain
C library and needs neither torch nor its headers."""

import os

import pytest

from spectral_convolution_amd import build


class _Done:
    returncode, stdout, stderr = 0, "", ""


@pytest.fixture
def linked(monkeypatch, tmp_path):
    """build() with the compilers replaced: the commands that ran, objects and outputs under tmp_path."""
    cmds = []

    def run(cmd, **_):
        cmds.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return _Done()

    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfno.so"))
    monkeypatch.setattr(build, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(build, "_hipcc", lambda: "hipcc")
    monkeypatch.setattr(build.subprocess, "run", run)
    return cmds


def test_without_torch_the_library_is_built(linked, monkeypatch, capsys):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.NATIVE) and "torch is not installed" in capsys.readouterr().err


def test_a_failing_extension_leaves_the_library(linked, monkeypatch):
    def fails(_):
        raise RuntimeError("g++ failed on binding.cpp")

    monkeypatch.setattr(build, "_native", fails)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build()
    assert os.path.exists(build.LIB)


def test_with_torch_both_are_built(linked):
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.NATIVE)
    assert len(linked) == len(build.SOURCES) + 2


def test_an_extension_that_does_not_load_says_why(monkeypatch):
    import sys

    import spectral_convolution_amd as fno
    from spectral_convolution_amd import _training as ops
    monkeypatch.setattr(ops, "_torch", None)
    monkeypatch.setitem(sys.modules, "spectral_convolution_amd._native", None)
    monkeypatch.delattr(fno, "_native", raising=False)
    with pytest.raises(RuntimeError, match="does not load: .*_native"):
        ops._t()
