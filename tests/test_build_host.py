"""The extension module of the row operators' calls: built for the PyTorch that is installed, and loaded for no other."""
import os
import subprocess

import pytest

from jagged_attention_recsys_gdpa_gb300 import _binding as B
from jagged_attention_recsys_gdpa_gb300 import build as build_mod


@pytest.fixture
def compilers(monkeypatch):
    """Stand-ins for nvcc and g++ that write what they are asked for: the commands, and those that shall fail."""
    commands, failing = [], set()

    def run(cmd, **kw):
        commands.append(cmd)
        name = os.path.basename(cmd[0])
        if name in failing:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write(name)
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build_mod.subprocess, "run", run)
    return commands, failing


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    for name in ("LIB", "HOST", "HOST_FOR"):
        monkeypatch.setattr(build_mod, name, str(tmp_path / os.path.basename(getattr(build_mod, name))))
    monkeypatch.setattr(build_mod, "BUILD", str(tmp_path))
    return tmp_path


@pytest.mark.parametrize("built", [None, "PyTorch 1.0, Python cpython-39"])
def test_a_module_for_another_pytorch_is_refused(monkeypatch, tmp_path, built):
    build_mod.build()
    monkeypatch.setattr(B, "_host", None)
    assert B.host() is not None
    monkeypatch.setattr(B, "_host", None)
    stamp = tmp_path / "_host.for"
    monkeypatch.setattr(build_mod, "HOST_FOR", str(stamp))
    if built is not None:
        stamp.write_text(built)
    with pytest.raises(RuntimeError, match="built for .*PyTorch"):
        B.host()


def test_a_module_for_another_pytorch_is_built_again_and_nothing_else(elsewhere, compilers):
    commands, _ = compilers
    build_mod.build()
    assert len(commands) == len(build_mod.SOURCES) + 2 and build_mod.host_misfit() == ""
    del commands[:]
    build_mod.build()
    assert commands == []
    (elsewhere / "_host.for").write_text("PyTorch 1.0, Python cpython-39")
    build_mod.build()
    assert [c[0] for c in commands] == ["g++"] and build_mod.host_misfit() == ""


def test_a_module_that_fails_leaves_the_library(elsewhere, compilers):
    """The error is raised, and attention and the paged cache have their library all the same."""
    commands, failing = compilers
    failing.add("g++")
    with pytest.raises(RuntimeError, match="host.cpp"):
        build_mod.build()
    assert (elsewhere / "libjattn.so").exists() and not (elsewhere / "_host.so").exists()
    del commands[:]
    failing.clear()
    build_mod.build()  # what is missing, and nothing else
    assert [c[0] for c in commands] == ["g++"] and (elsewhere / "_host.so").exists()
