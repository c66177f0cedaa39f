"""What build() compiles, and when (the compilers are replaced: no GPU, no nvcc)."""
import importlib
import os
import types

import pytest
import torch

import chunked_gated_delta_10_gb300 as kda

build = importlib.import_module("chunked_gated_delta_10_gb300.build")


@pytest.fixture
def ran(monkeypatch, tmp_path):
    """The commands that build() ran, in a folder of its own; each writes its output file, or fails where `ran.fails` is in it."""
    commands = types.SimpleNamespace(list=[], fails=None)

    def run(cmd, **_):
        commands.list.append(cmd)
        if commands.fails and any(commands.fails in x for x in cmd):
            return types.SimpleNamespace(returncode=1, stdout="", stderr="it fails")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("x")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(build.subprocess, "run", run)
    for name, path in (("OBJ", "_build"), ("LIB_DIR", "lib"), ("LIB", "lib/a.so"), ("SERVE", "lib/b.so")):
        monkeypatch.setattr(build, name, str(tmp_path / path))
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    monkeypatch.setattr(build, "_serve_missing", lambda: None)
    return commands


def outputs(commands):
    return sorted(os.path.basename(c[c.index("-o") + 1]).split(".tmp")[0] for c in commands.list)


def test_everything_once(ran):
    build.build()
    sources = [os.path.basename(s) + ".o" for s in build._sources()]
    assert outputs(ran) == sorted(sources + ["serve_binding.o", "a.so", "b.so"])
    ran.list.clear()
    build.build()
    assert not ran.list


def test_another_pytorch_makes_the_module_anew(ran, monkeypatch):
    build.build()
    ran.list.clear()
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    build.build()
    assert outputs(ran) == ["b.so", "serve_binding.o"]
    ran.list.clear()
    build.build()
    assert not ran.list


def test_without_the_modules_headers_the_library_is_built(ran, monkeypatch):
    build.build()
    monkeypatch.setattr(build, "_serve_missing", lambda: "/nowhere/Python.h")
    ran.list.clear()
    with pytest.warns(UserWarning, match="Python.h"):
        assert build.build(force=True) == build.LIB
    assert "a.so" in outputs(ran) and "b.so" not in outputs(ran) and "serve_binding.o" not in outputs(ran)
    assert not os.path.exists(build.SERVE)  # what was there belongs to another PyTorch
    monkeypatch.setattr(kda, "SERVE", build.SERVE)
    monkeypatch.setattr(kda, "_serve_module", None)
    monkeypatch.setattr(kda, "load", lambda: None)
    with pytest.raises(RuntimeError, match="not built"):
        kda._serve()


def test_a_module_that_does_not_compile_is_an_error_beside_a_whole_library(ran):
    ran.fails = "serve_binding"
    with pytest.raises(RuntimeError, match="it fails"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.SERVE)
    ran.fails = None
    ran.list.clear()
    build.build()
    assert outputs(ran) == ["b.so", "serve_binding.o"]


def test_what_is_missing(monkeypatch, tmp_path):
    """A PyTorch without CUDA, or without its headers; a Python without its own."""
    assert build._serve_missing() is None
    with monkeypatch.context() as m:
        m.setattr(torch, "__file__", str(tmp_path / "__init__.py"))
        assert build._serve_missing().startswith(str(tmp_path))
    with monkeypatch.context() as m:
        m.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
        assert build._serve_missing() == str(tmp_path / "Python.h")
    with monkeypatch.context() as m:
        m.setattr(torch.version, "cuda", None)
        assert "CUDA" in build._serve_missing()
