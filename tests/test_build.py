"""The build: the C library needs hipcc alone (no GPU needed; nothing is compiled here, commands are recorded)."""
import os
import subprocess
import sys

import pytest

from bit_quantized_gemm_amd import build as b


@pytest.fixture
def recorded(monkeypatch, tmp_path):
    """build() with its output in tmp_path and its commands in a list; each writes what it says it writes."""
    commands = []

    def run(cmd, **k):
        commands.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libatom.so"))
    monkeypatch.setattr(b, "SHORT", str(tmp_path / "_short.so"))
    return commands


def linked(commands):
    return [c for c in commands if c[0] == b.HIPCC and "-shared" in c]


def test_both_libraries(recorded):
    pytest.importorskip("torch")
    if not b.shutil.which("g++"):
        pytest.skip("no g++")
    assert b.build() == b.LIB and os.path.exists(b.LIB) and os.path.exists(b.SHORT)
    assert len(linked(recorded)) == 1 and len(recorded) == len(b.SOURCES) + 2


@pytest.mark.parametrize("missing", ["torch", "compiler", "headers"])
def test_the_c_library_without_the_extension(recorded, monkeypatch, capsys, missing):
    """What only the extension module needs is missing: the C library is linked, an older module does not stay, and stderr says why."""
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)                 # its import fails
    else:
        pytest.importorskip("torch")
    if missing == "compiler":
        monkeypatch.delenv("CXX", raising=False)
        monkeypatch.setattr(b.shutil, "which", lambda name: None)
    if missing == "headers":
        import sysconfig
        monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": "/nowhere"})
    with open(b.SHORT, "w"):
        pass
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert len(linked(recorded)) == 1
    assert not os.path.exists(b.SHORT)
    assert "not built" in capsys.readouterr().err


def test_a_module_that_does_not_compile_is_an_error(recorded, monkeypatch):
    """Behind the link: the C library is there all the same."""
    pytest.importorskip("torch")

    def fail():
        raise RuntimeError("failed for short_calls.cpp")
    monkeypatch.setattr(b, "_build_short", fail)
    with pytest.raises(RuntimeError, match="short_calls"):
        b.build()
    assert os.path.exists(b.LIB) and len(linked(recorded)) == 1
