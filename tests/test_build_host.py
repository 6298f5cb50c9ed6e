"""The C library needs nvcc only: a machine without torch, or without what its Python module needs, still
builds libttq.so."""

import importlib.util
import os
import sys

import pytest

from online_activation_aware_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build that compiles nothing: the library's commands are recorded and leave empty files."""
    ran = []

    def run(cmd, **kw):
        ran.append(os.path.basename(cmd[0]))
        open(cmd[cmd.index("-o") + 1], "w").close()

        class Done:
            returncode, stdout, stderr = 0, "", ""
        return Done

    monkeypatch.setattr(build, "LIB", str(tmp_path / "libttq.so"))
    monkeypatch.setattr(build, "HOST", str(tmp_path / "_host.so"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_without_torch_the_library_is_built(tree, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setitem(sys.modules, "torch", None)      # (importing it fails)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.HOST)
    assert build.build() == build.LIB      # nothing left to do


def test_a_module_that_does_not_compile_does_not_hide_the_library(tree, monkeypatch):
    def broken(*a, **kw):
        raise RuntimeError("the host compiler failed")

    monkeypatch.setattr(build, "build_host", broken)
    with pytest.raises(RuntimeError, match="host compiler"):
        build.build()
    assert os.path.exists(build.LIB)
