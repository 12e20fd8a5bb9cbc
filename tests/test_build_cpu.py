"""What build() needs: hipcc for the library, PyTorch's headers and a host
compiler for the compiled Python calls only (no compiler runs here)."""
import os

import pytest

from mixed_precision_quantized_act_amd import build as b


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The command lines that build() runs; each leaves its output empty."""
    seen = []

    def run(cmd):
        seen.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "hipcc", lambda: "/opt/rocm/bin/hipcc")
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path / "obj"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libqact.so"))
    monkeypatch.setattr(b, "CALL", str(tmp_path / "_call.so"))
    return seen


def _calls(commands):
    return [c for c in commands if any(a.endswith("pycall.cpp") for a in c)]


def test_with_everything(commands, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(b.shutil, "which", lambda name: "/usr/bin/" + name)
    b.build(verbose=False)
    assert os.path.exists(b.LIB) and os.path.exists(b.CALL)
    assert len(_calls(commands)) == 1 and len(commands) == len(b.SOURCES) + 2


@pytest.mark.parametrize("missing", ["torch", "compiler"])
def test_the_library_alone(commands, monkeypatch, capsys, missing):
    if missing == "torch":
        monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.setattr(b.shutil, "which", lambda name: None)
    assert b.build(verbose=False) == b.LIB
    assert os.path.exists(b.LIB) and not os.path.exists(b.CALL)
    assert not _calls(commands) and len(commands) == len(b.SOURCES) + 1
    assert "_call.so" in capsys.readouterr().out


def test_calls_that_do_not_compile_leave_the_library(commands, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setattr(b.shutil, "which", lambda name: "/usr/bin/" + name)
    run = b._run

    def fails(cmd):
        if _calls([cmd]):
            raise RuntimeError("compiler failed")
        run(cmd)

    monkeypatch.setattr(b, "_run", fails)
    with pytest.raises(RuntimeError):
        b.build(verbose=False)
    assert os.path.exists(b.LIB) and not os.path.exists(b.CALL)


@pytest.mark.parametrize("missing", ["compiler", "success"])
def test_calls_of_an_older_library_do_not_stay(commands, monkeypatch, missing):
    """A _call.so that is there was built against the functions of the library that is replaced."""
    pytest.importorskip("torch")
    monkeypatch.setattr(b.shutil, "which", lambda name: None if missing == "compiler" else "/usr/bin/" + name)
    with open(b.CALL, "w") as f:
        f.write("older")
    run = b._run

    def fails(cmd):
        if _calls([cmd]):
            raise RuntimeError("compiler failed")
        run(cmd)

    if missing == "success":
        monkeypatch.setattr(b, "_run", fails)
        with pytest.raises(RuntimeError):
            b.build(verbose=False)
    else:
        b.build(verbose=False)
    assert os.path.exists(b.LIB) and not os.path.exists(b.CALL)
