"""The build: the C library needs hipcc alone (no GPU needed; nothing is compiled here, commands are recorded)."""
import os
import subprocess
import sys

import pytest

import bit_quantized_gemm_amd as bq
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
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": "/nowhere"})
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


# ---- the extension module holds torch's insides: it is used with the torch and the Python that it was built with alone
@pytest.fixture
def module():
    pytest.importorskip("torch")
    if not os.path.exists(bq.lib_path()):
        pytest.skip("libatom.so not built (python -m bit_quantized_gemm_amd.build)")
    bq.load_library()
    if bq._SHORT is None:
        pytest.skip("the extension module is not built")
    return bq._SHORT


def test_the_module_names_what_it_was_built_for(module):
    import torch
    assert module.built_for == bq._built_for() and torch.__version__ in module.built_for and "cpython" in module.built_for
    assert os.path.basename(module.__file__) == os.path.basename(b.SHORT) == "_short" + b.sysconfig.get_config_var("EXT_SUFFIX")


@pytest.mark.parametrize("other", ["version", "build", "python"])
def test_a_module_of_another_torch_is_left_alone(module, monkeypatch, other):
    """None, with a warning that names both; what was bound stays as it is."""
    import torch
    if other == "version":
        monkeypatch.setattr(torch, "__version__", "9.9.9")
    elif other == "build":
        monkeypatch.setattr(torch.version, "git_version", "0" * 40)
    else:
        monkeypatch.setattr(bq.sys, "implementation", type("I", (), {"cache_tag": "cpython-399"}))
    with pytest.warns(RuntimeWarning, match="was built for"):
        assert bq._bind_short(bq._LIB, ("atom_linear_mxfp4",)) is None


def test_a_module_that_says_nothing_is_left_alone(module, monkeypatch):
    monkeypatch.delattr(module, "built_for")
    with pytest.warns(RuntimeWarning, match="unknown torch"):
        assert bq._bind_short(bq._LIB, ()) is None
