"""The extension module is built again for another PyTorch or Python, and says so when it meets one
that it was not built for."""
import builtins
import subprocess

import pytest
import torch

import nvfp4_block_scaled_17_b200 as nv
from nvfp4_block_scaled_17_b200 import _build


@pytest.fixture
def built():
    _build.build()


@pytest.fixture
def compilers(built, monkeypatch):
    """The commands that would have been run."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        raise subprocess.CalledProcessError(1, cmd)
    monkeypatch.setattr(_build.subprocess, "run", run)
    return ran


def test_up_to_date_is_left(compilers):
    assert _build.build_binding() == _build.BINDING_PATH
    assert compilers == []


@pytest.mark.parametrize("change", ["torch", "abi", "python"])
def test_another_environment_builds_again(compilers, monkeypatch, change):
    if change == "torch":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif change == "abi":
        abi = torch.compiled_with_cxx11_abi()
        monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: not abi)
    else:
        monkeypatch.setattr(_build.sys, "version", "2.7.18")
    with pytest.raises(subprocess.CalledProcessError):
        _build.build_binding()
    assert len(compilers) == 1 and _build.BINDING_SRC in compilers[0]


def test_another_torch_at_run_time(built, monkeypatch):
    monkeypatch.setattr(nv, "_bound", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with pytest.raises(RuntimeError, match="built for PyTorch .*0.0.1.*build it again"):
        nv._calls()


def test_import_errors_say_why(built, monkeypatch):
    real = builtins.__import__

    def refuse(name, globals=None, locals=None, fromlist=(), level=0):
        if fromlist and "_binding" in fromlist:
            raise ImportError("undefined symbol: something")
        return real(name, globals, locals, fromlist, level)
    monkeypatch.setattr(nv, "_bound", None)
    monkeypatch.setattr(builtins, "__import__", refuse)
    with pytest.raises(RuntimeError, match="undefined symbol: something"):
        nv._calls()
