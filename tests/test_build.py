"""CPU: the build makes the library whatever becomes of the marshalling module, and the module that is loaded is one
that was built for this Python, this torch and these sources."""
import os
import subprocess

import pytest

import gqa_decode_attention_04_b200 as gq
from gqa_decode_attention_04_b200 import build as B


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """The build's outputs go to a folder of their own, with nothing in it yet; commands are recorded, and make
    their -o file unless they are a C++ compiler's and `broken` is set."""
    state = {"commands": [], "broken": False}
    monkeypatch.setattr(B, "HERE", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libgqa_decode.so"))
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


def modules():
    return sorted(n for n in os.listdir(B.HERE) if n.startswith("_fastcall"))


def test_the_module_is_rebuilt_for_another_torch_python_or_source(tree, monkeypatch, tmp_path):
    import torch
    B.build()
    (first,) = modules()
    n = len(tree["commands"])
    B.build_fastcall()
    assert len(tree["commands"]) == n  # nothing to do
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    B.build_fastcall()
    (second,) = modules()
    monkeypatch.setattr(B.sysconfig, "get_config_var", lambda name: "other")
    B.build_fastcall()
    (third,) = modules()
    header = tmp_path / "include"
    header.mkdir()
    (header / "gqa_int4.h").write_text("another argument\n")
    monkeypatch.setattr(B, "INCLUDE", str(header))
    B.build_fastcall()
    (fourth,) = modules()
    assert len({first, second, third, fourth}) == 4
    assert len(tree["commands"]) == n + 3


def test_a_module_built_for_others_is_not_loaded(monkeypatch):
    lib = gq.load_library()
    monkeypatch.setattr(gq, "_fast", None)
    gq._load_fast(lib)
    assert gq._fast is not None
    import torch
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    monkeypatch.setattr(gq, "_fast", None)
    gq._load_fast(lib)
    assert gq._fast is None


def test_the_module_takes_its_entry_points_types_from_the_headers():
    """A call whose arguments no longer are the entry point's does not compile."""
    with open(B.FAST_SOURCE) as f:
        text = f.read()
    assert "(*)(" not in text.replace("reinterpret_cast<void (*)()>", "")
    for name in ("gqa_rope_kv_append", "gqa_rope_kv_append_fp8", "gqa_rope_kv_append_int4", "gqa_kv_quantize_int4",
                 "gqa_kv_dequantize_int4", "gqa_paged_decode_attn_int4", "gqa_paged_multi_query_attn_int4", "gqa_decode_step_int4"):
        assert f"ENTRY({name}," in text
