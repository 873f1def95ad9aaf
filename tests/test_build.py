"""The build of the library and of the Python binding's native part: what is built for what,
and what needs what (host only)."""

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
