"""CPU: the build makes the library whatever becomes of the marshalling module."""
import os
import subprocess

import pytest

from gqa_decode_attention_04_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's outputs go to a folder of their own, with nothing in it yet; commands are recorded, and make
    their -o file unless they are a C++ compiler's and `broken` is set."""
    state = {"commands": [], "broken": False}
    monkeypatch.setattr(B, "HERE", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libgqa_decode.so"))
    monkeypatch.setattr(B, "FAST", str(tmp_path / "_fastcall.so"))
    monkeypatch.setenv("CXX", "some-g++")

    def run(cmd, **kw):
        state["commands"].append(cmd)
        if cmd[0] == "some-g++" and state["broken"]:
            if state["broken"] == "missing":
                raise FileNotFoundError("some-g++")
            return subprocess.CompletedProcess(cmd, 1, "", "no headers")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    return state


@pytest.mark.parametrize("how", ["fails", "missing"])
def test_the_library_is_built_without_a_cpp_compiler(tree, how, capsys):
    tree["broken"] = how
    assert B.build(force=True) == B.LIB and os.path.exists(B.LIB)
    assert "without the marshalling module" in capsys.readouterr().err
    assert not any(n.startswith("_fastcall") for n in os.listdir(B.HERE))


def test_a_library_that_fails_is_an_error(tree, monkeypatch):
    def fails(cmd, **kw):
        return subprocess.CompletedProcess(cmd, 1, "", "")
    monkeypatch.setattr(subprocess, "run", fails)
    with pytest.raises(RuntimeError, match="nvcc"):
        B.build(force=True)
