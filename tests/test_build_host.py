"""What build() compiles, with a stand-in for the compilers: they make empty files."""
import os
import subprocess
import types

import pytest

from rank_adapter_apply_gb300 import build as build_mod


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Commands run, in an empty build folder."""
    commands = []

    def run(cmd, **kw):
        commands.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")
    monkeypatch.setattr(subprocess, "run", run)
    out = str(tmp_path / "_build")
    monkeypatch.setattr(build_mod, "BUILD", out)
    monkeypatch.setattr(build_mod, "LIB", os.path.join(out, "librank_adapter_apply.so"))
    monkeypatch.setattr(build_mod, "TENSOR_CALLS", os.path.join(out, "_tensor_calls.so"))
    return commands


def _without_torch(monkeypatch):
    import importlib.util
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def test_library_is_built_without_torch(monkeypatch, made):
    """The C library does not need torch, and neither does building it; with torch the module is built afterwards."""
    with monkeypatch.context() as m:
        _without_torch(m)
        lib = build_mod.build()
        assert os.path.exists(lib) and len(made) == len(build_mod.SOURCES) + 1
        assert not os.path.exists(build_mod.TENSOR_CALLS)
    made.clear()
    build_mod.build()
    assert len(made) == 1 and os.path.exists(build_mod.TENSOR_CALLS)


def test_module_is_built_again_for_another_torch(monkeypatch, made, tmp_path):
    """Nothing to do a second time; another torch at the same place means another module, and nothing else."""
    torch = tmp_path / "torch"
    torch.mkdir()
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("__version__ = '2.9.1'\n")
    import importlib.util
    find = importlib.util.find_spec
    spec = types.SimpleNamespace(origin=str(torch / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec if name == "torch" else find(name, *a))
    build_mod.build()
    assert len(made) == len(build_mod.SOURCES) + 2
    made.clear()
    build_mod.build()
    assert not made
    old = os.path.getmtime(torch / "version.py") - 1000
    (torch / "version.py").write_text("__version__ = '2.11.0'\n")
    os.utime(torch / "version.py", (old, old))
    build_mod.build()
    assert len(made) == 1 and made[0][made[0].index("-o") - 1] == build_mod.TENSOR_CALLS_SOURCE
    made.clear()
    build_mod.build()
    assert not made
