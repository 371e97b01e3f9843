"""What the build does where torch is missing or has changed."""
import importlib.util
import os
import subprocess

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build module over outputs of its own; .ran holds the commands that it would have run."""
    from bit_quantized_moe_routed_b200 import build as b
    monkeypatch.setattr(b, "CALLS_SO", str(tmp_path / "_torch_calls.so"))
    monkeypatch.setattr(b, "CALLS_STAMP", str(tmp_path / "stamp"), raising=False)
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    b.ran = ran
    return b


def hide_torch(monkeypatch):
    import builtins
    find, imp = importlib.util.find_spec, builtins.__import__

    def no_torch(name, *a, **kw):
        if name == "torch":
            raise ImportError("No module named 'torch'")
        return imp(name, *a, **kw)
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(builtins, "__import__", no_torch)


def test_the_library_builds_without_torch(build, monkeypatch, capsys):
    hide_torch(monkeypatch)
    build._build_calls(False, False)
    assert not build.ran and not os.path.exists(build.CALLS_SO)
    assert "torch is not installed" in capsys.readouterr().err


def test_the_library_builds_without_headers(build, monkeypatch, capsys):
    paths = build.sysconfig.get_paths()
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: dict(paths, include="/nowhere"))
    build._build_calls(False, False)
    assert not build.ran and "/nowhere/Python.h" in capsys.readouterr().err


def test_another_torch_or_python_builds_the_calls_again(build, monkeypatch):
    build._build_calls(False, False)
    assert len(build.ran) == 1 and os.path.exists(build.CALLS_SO)
    build._build_calls(False, False)
    assert len(build.ran) == 1                      # up to date
    with monkeypatch.context() as m:
        m.setattr(build.sys, "version", "another")
        build._build_calls(False, False)
        assert len(build.ran) == 2
    build._build_calls(False, False)
    assert len(build.ran) == 3
    build._build_calls(True, False)
    assert len(build.ran) == 4


def test_another_torch_version_builds_the_calls_again(build, monkeypatch, tmp_path):
    build._build_calls(False, False)
    import torch
    root = tmp_path / "torch"
    (root / "include" / "ATen").mkdir(parents=True)
    (root / "include" / "ATen" / "ATen.h").write_text("")
    (root / "version.py").write_text("__version__ = 'another'\n")
    spec = importlib.util.find_spec("torch")

    class Moved:
        origin = str(root / "__init__.py")
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: Moved if name == "torch" else spec)
    monkeypatch.setattr(torch, "__file__", Moved.origin)
    build._build_calls(False, False)
    assert len(build.ran) == 2 and str(root / "lib") in build.ran[1]
