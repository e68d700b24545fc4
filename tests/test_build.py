"""What build() compiles and keeps, with the compilers faked: the library does not depend on the binding's extension."""
import os
import subprocess
import time

import pytest

from gqa_split_kv_gb300 import build as b


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """Compilers that write their output file, and a PyTorch folder; state.fails: substrings of commands that fail."""
    class State:
        ran, fails, torch = [], (), str(tmp_path / "torch")

    def run(cmd):
        State.ran.append(cmd)
        if any(f in " ".join(cmd) for f in State.fails):
            return subprocess.CompletedProcess(cmd, 1, "", "no")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    os.makedirs(os.path.join(State.torch, "include", "ATen", "core"))
    open(os.path.join(State.torch, "include", "ATen", "core", "Tensor.h"), "w").close()
    with open(os.path.join(State.torch, "version.py"), "w") as f:
        f.write("__version__ = '1'")
    include = tmp_path / "python"
    include.mkdir()
    (include / "Python.h").touch()
    monkeypatch.setattr(b, "_run", run)
    monkeypatch.setattr(b, "nvcc_path", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(include)})
    find = b.importlib.util.find_spec
    spec = type("Spec", (), {"submodule_search_locations": property(lambda self: [State.torch])})()
    monkeypatch.setattr(b.importlib.util, "find_spec",
                        lambda name, *a: (spec if State.torch else None) if name == "torch" else find(name, *a))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "EXT", str(tmp_path / "ext.so"))
    monkeypatch.setattr(b, "EXT_STAMP", str(tmp_path / "_build" / "stamp"), raising=False)
    State.include = include
    return State


def made():
    return os.path.exists(b.LIB), os.path.exists(b.EXT)


def test_both_once(fake):
    assert b.build() == b.LIB and made() == (True, True) and len(fake.ran) == len(b.SOURCES) + 2
    b.build()
    assert len(fake.ran) == len(b.SOURCES) + 2
    b.build(force=True)
    assert len(fake.ran) == 2 * (len(b.SOURCES) + 2)


@pytest.mark.parametrize("lost", ["torch", "torch headers", "Python.h"])
def test_the_library_alone(fake, lost, capsys):
    if lost == "torch":
        fake.torch = None
    elif lost == "torch headers":
        os.remove(os.path.join(fake.torch, "include", "ATen", "core", "Tensor.h"))
    else:
        (fake.include / "Python.h").unlink()
    assert b.build() == b.LIB and made() == (True, False)
    assert "extension is not built" in capsys.readouterr().out
    n = len(fake.ran)
    b.build()
    assert len(fake.ran) == n


def test_a_failing_extension_leaves_the_library(fake):
    fake.fails = ("binding_ext.cpp",)
    with pytest.raises(RuntimeError, match="extension"):
        b.build()
    assert made() == (True, False)


def test_a_failing_library_says_so(fake):
    fake.fails = ("cache_ops.cu",)
    with pytest.raises(RuntimeError, match="libdecode_attn.so"):
        b.build()
    assert not made()[0]


def test_another_pytorch_makes_the_extension_anew(fake):
    b.build()
    fake.ran.clear()
    time.sleep(0.01)
    with open(os.path.join(fake.torch, "version.py"), "w") as f:
        f.write("__version__ = '2'")
    b.build()
    assert len(fake.ran) == 1 and "binding_ext.cpp" in " ".join(fake.ran[0])
    b.build()
    assert len(fake.ran) == 1
