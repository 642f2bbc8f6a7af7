"""The build's steps, with the compilers replaced by stand-ins."""

import importlib.util
import os
import subprocess
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module by its file, as `python moe_grouped_mlp_amd/build.py`
    runs it, in a folder of its own."""
    spec = importlib.util.spec_from_file_location("build_alone", os.path.join(ROOT, "moe_grouped_mlp_amd", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    for name, file in (("HERE", ""), ("BUILD", "_build"), ("LIB", "lib.so"), ("CALL", "_call.so")):
        monkeypatch.setattr(b, name, str(tmp_path / file))
    monkeypatch.setattr(b, "HIPCC", sys.executable)   # a file that exists

    def run(cmd, **kw):
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stderr="", stdout="")

    monkeypatch.setattr(subprocess, "run", run)
    return b


def test_library_builds_without_torch(build, monkeypatch, capsys):
    """The C ABI needs no torch; the Python binding's compiled part does, and an
    older one is not left beside a new library."""
    for name in [n for n in sys.modules if n.split(".")[0] == "torch"]:
        monkeypatch.delitem(sys.modules, name)
    monkeypatch.setitem(sys.modules, "torch", None)   # as where it is not installed
    open(build.CALL, "w").close()
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALL)
    assert "torch" in capsys.readouterr().out


def test_both_are_built_with_torch(build, capsys):
    build.build()
    assert os.path.exists(build.LIB) and os.path.exists(build.CALL)
    out = capsys.readouterr().out
    assert build.LIB in out and build.CALL in out
