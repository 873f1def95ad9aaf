"""The build of the library and of the Python binding's native part: what is built for what,
and what needs what (host only)."""

import sys
import sysconfig

import pytest

import paged_head_latent_mla_b200 as M
from paged_head_latent_mla_b200 import _build


def test_the_native_part_is_named_after_python_and_torch(monkeypatch):
    import torch

    here = _build.marshal_path()
    assert torch.__version__ in here and sysconfig.get_config_var("SOABI") in here and here.endswith(".so")
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    other = _build.marshal_path()
    assert other != here
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-299")
    assert _build.marshal_path() not in (here, other)


def test_the_native_part_of_another_torch_is_not_loaded(monkeypatch):
    """Not even where its file is there and would load."""
    import torch

    _build.build()
    monkeypatch.setattr(M, "_helpers", None)
    assert M._native().device() >= -1  # this torch's
    monkeypatch.setattr(M, "_helpers", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(RuntimeError, match="missing or stale"):
        M._native()


def test_the_native_part_of_another_torch_does_not_count_as_built(monkeypatch):
    import torch

    _build.build()
    ran = []
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or _Done())
    monkeypatch.setattr(_build.os, "replace", lambda a, b: None)
    _build.build_marshal()
    assert not ran
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    _build.build_marshal()
    assert len(ran) == 1 and "0.0.1+other" in ran[0][ran[0].index("-o") + 1]


class _Done:
    returncode, stdout, stderr = 0, "", ""


def _recorded(monkeypatch):
    """Compilers that only record that they were called."""
    ran = []
    monkeypatch.setattr(_build.subprocess, "run", lambda cmd, **kw: ran.append(cmd[0].split("/")[-1]) or _Done())
    monkeypatch.setattr(_build.os, "replace", lambda a, b: None)
    return ran


def test_the_library_is_built_without_torch(monkeypatch, capsys):
    ran = _recorded(monkeypatch)
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: None)
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it fails
    assert _build.build(force=True) == _build.LIB
    assert ran == ["nvcc"] and "torch is not installed" in capsys.readouterr().err


def test_the_library_alone_on_request(monkeypatch):
    ran = _recorded(monkeypatch)
    monkeypatch.setitem(sys.modules, "torch", None)
    _build.build(force=True, library_only=True)
    assert ran == ["nvcc"]


def test_a_binding_that_does_not_compile_leaves_the_library(monkeypatch):
    """(no Python.h, for instance)"""
    ran = _recorded(monkeypatch)
    done = _build.subprocess.run

    def run(cmd, **kw):
        out = done(cmd, **kw)
        if cmd[0] == "g++":
            out.returncode, out.stderr = 1, "Python.h: No such file"
        return out

    monkeypatch.setattr(_build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="Python.h"):
        _build.build(force=True)
    assert ran == ["nvcc", "g++"]
