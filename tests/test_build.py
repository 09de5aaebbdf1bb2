"""The build: the library needs nvcc only; the binding's native argument checks are built where torch
is, against that torch, and are optional."""
import os
import subprocess
import types

import pytest

import __graft_entry__


@pytest.fixture
def builder(tmp_path, monkeypatch):
    """The build module with its products of the binding in a folder of their own."""
    b = __graft_entry__._load_builder()
    monkeypatch.setattr(b, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(b, "OBJ", str(tmp_path / "obj"))
    return b


def compiler(builder, monkeypatch, rc=0):
    """Stands in for the compiler: writes what it is asked to write; returns its calls."""
    calls = []

    def run(cmd, **kw):
        calls.append(cmd)
        if rc == 0:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=rc, stderr="no Python.h", stdout="")

    monkeypatch.setattr(builder, "subprocess", types.SimpleNamespace(run=run))
    return calls


def test_the_library_builds_without_torch(builder, monkeypatch):
    monkeypatch.setattr(builder.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setattr(builder, "_build_lib", lambda force, v: builder.LIB)
    calls = compiler(builder, monkeypatch)
    assert builder.build() == builder.LIB
    assert builder.build(force=True) == builder.LIB
    assert not calls and not os.path.exists(builder.BIND)


@pytest.mark.parametrize("missing", ["headers", "compiler"])
def test_the_library_builds_without_what_the_checks_need(builder, monkeypatch, capsys, missing):
    monkeypatch.setattr(builder, "_build_lib", lambda force, v: builder.LIB)
    open(builder.BIND, "w").close()  # of an earlier torch: must not be left to be loaded
    if missing == "headers":
        compiler(builder, monkeypatch, rc=1)
    else:
        monkeypatch.setenv("CXX", "/nonexistent/compiler")
    assert builder.build() == builder.LIB
    assert not os.path.exists(builder.BIND) and "_bind.so is not built" in capsys.readouterr().err


def test_the_checks_are_built_again_where_torch_changes(builder, monkeypatch):
    calls = compiler(builder, monkeypatch)
    assert builder._build_bind() and len(calls) == 1
    assert builder._build_bind() and len(calls) == 1
    assert builder._build_bind(force=True) and len(calls) == 2
    monkeypatch.setattr(builder, "_bind_stamp", lambda d: "another torch")
    assert builder._build_bind() and len(calls) == 3
    assert builder._build_bind() and len(calls) == 3


def test_the_binding_works_without_the_native_checks():
    # without _bind the same checks are made in Python
    code = ("import sys; sys.modules['weight_sequence_layers_b200._bind'] = None\n"
            "import torch, weight_sequence_layers_b200 as ttt\n"
            "c = ttt.make_norm_config(1, 1, 2, 8, 'f32')\n"
            "try: ttt.ttt_norm_fwd(c, torch.zeros(16), None, None, None, torch.zeros(16))\n"
            "except ValueError as e: assert 'CUDA' in str(e), e\n"
            "else: raise SystemExit('not refused')\n"
            "assert ttt._modules[1] is None\n")
    r = subprocess.run([os.sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=__graft_entry__.ROOT)
    assert r.returncode == 0, r.stderr
