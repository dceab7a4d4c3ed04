"""What the build makes where torch or its headers are missing (commands recorded, nothing compiled)."""
import os

import pytest

from persistent_transformer_megakernel_gb300 import build as b


@pytest.fixture
def commands(monkeypatch, tmp_path):
    ran = []

    def run(cmd):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "OUT_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmk.so"))
    monkeypatch.setattr(b, "MODULE", str(tmp_path / "_mktorch.so"))
    return ran


def test_both(commands):
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.MODULE)
    assert len(commands) == len(b.SOURCES) + 3


def _no_torch():
    raise ImportError("No module named 'torch'")


def test_the_library_without_torch(commands, monkeypatch):
    monkeypatch.setattr(b, "_torch_dir", _no_torch)
    open(b.MODULE, "w").close()                             # of an earlier build
    with pytest.raises(RuntimeError, match="_mktorch.so .*is not.*torch"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.MODULE)


def test_the_library_where_the_module_does_not_compile(commands, monkeypatch):
    run = b._run

    def refuse(cmd):
        if cmd[0] == "g++":
            raise RuntimeError("command failed: Python.h: No such file or directory")
        return run(cmd)
    monkeypatch.setattr(b, "_run", refuse)
    with pytest.raises(RuntimeError, match="Python.h"):
        b.build()
    assert os.path.exists(b.LIB)


def test_the_library_alone(commands, monkeypatch):
    monkeypatch.setattr(b, "_torch_dir", _no_torch)
    assert b.build(module=False) == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.MODULE)
    assert len(commands) == len(b.SOURCES) + 1 and all(os.path.basename(c[0]) == "nvcc" for c in commands)
