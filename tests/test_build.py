"""The build script: the C library needs no torch, the native part of the binding does."""

import importlib.util
import os

import pytest

from fp8_fine_grained_online_amd import build as B


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """A build into a folder of its own; commands are noted, not run, and leave an empty output."""
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(B, "_run", run)
    for name, file in (("BUILD_DIR", "_build"), ("LIB_PATH", "libfp8q.so"), ("BINDING_PATH", "_binding.so"),
                       ("PROBE_DIR", "none")):
        monkeypatch.setattr(B, name, str(tmp_path / file))
    return ran


def test_library_alone_without_torch(commands, monkeypatch, capsys):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert B.build() == B.LIB_PATH
    assert os.path.exists(B.LIB_PATH) and not os.path.exists(B.BINDING_PATH)
    assert "torch is not installed" in capsys.readouterr().err


def test_binding_with_torch(commands, capsys):
    B.build()
    assert os.path.exists(B.LIB_PATH) and os.path.exists(B.BINDING_PATH)
    assert all(cmd[0] == B.HIPCC for cmd in commands)  # one compiler for everything
    assert not capsys.readouterr().err


def test_missing_headers_are_named(monkeypatch, tmp_path):
    monkeypatch.setattr(B.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert "Python.h" in B.binding_needs()
