"""What build() does again, and what it does without PyTorch (nothing is compiled here: the
commands are noted and leave empty files)."""
import importlib.metadata
import os
import sys

import pytest

from dense_tensor_decomposition_gb300 import _build


@pytest.fixture
def commands(tmp_path, monkeypatch):
    done = []

    def note(cmd, what):
        done.append(what)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return type("Result", (), {"returncode": 0, "stderr": ""})

    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libmttkrp.so"))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(_build, "_run", note)
    return done


def test_everything_once(commands):
    pytest.importorskip("torch")
    assert not _build.up_to_date()
    _build.build()
    assert _build.up_to_date() and os.path.exists(_build.LIB) and os.path.exists(_build.BINDING)
    assert "linking the library" in commands and "linking the binding" in commands
    count = len(commands)
    _build.build()
    assert len(commands) == count


def test_another_pytorch(commands, monkeypatch):
    """The library stays, the module that would not load is built again."""
    pytest.importorskip("torch")
    _build.build()
    commands.clear()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.1")
    assert not _build.up_to_date()
    _build.build()
    assert commands == [f"compiling {_build._binding_source()}", "linking the binding"]
    assert _build.up_to_date()


def test_without_pytorch(commands, monkeypatch):
    """The C library needs no PyTorch, and neither does building it."""
    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)

    monkeypatch.setattr(importlib.metadata, "version", missing)
    monkeypatch.setitem(sys.modules, "torch", None)             # import torch raises
    _build.build()
    assert "linking the library" in commands and "linking the binding" not in commands
    assert _build.up_to_date()
