"""The INT8 path's host module depends on the layouts of one torch and one Python: it is used
only with those it was built for.  Needs no device."""
import os
import sysconfig

import torch

import block_scaled_precision_nvfp4_b200 as nv
from block_scaled_precision_nvfp4_b200 import _build

FAST = ("fast_gemm", "fast_grouped", "fast_quantize", "fast_topk")


def _used():
    return {getattr(nv._Host(), f) is not nv._no_fast_call for f in FAST}


def test_the_module_of_this_torch_is_used():
    path = _build.build_host_calls()
    assert os.path.exists(path) and _used() == {True}


def test_a_module_built_for_another_torch_is_not_used(monkeypatch):
    built = _build.build_host_calls()
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    assert _used() == {False}
    assert _build.host_calls_path() != built


def test_a_module_built_for_another_abi_or_python_is_not_used(monkeypatch):
    built = _build.build_host_calls()
    with monkeypatch.context() as m:
        m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", not torch._C._GLIBCXX_USE_CXX11_ABI)
        assert _used() == {False} and _build.host_calls_path() != built
    get = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-00-other" if n == "SOABI" else get(n))
    assert _used() == {False} and _build.host_calls_path() != built


def test_the_build_goes_on_without_the_module(monkeypatch, capsys):
    """The module needs torch's C++ headers; the calls do not need the module."""
    import subprocess
    import __graft_entry__

    def fails(force=False):
        raise subprocess.CalledProcessError(1, ["g++"])
    monkeypatch.setattr(_build, "build_host_calls", fails)
    __graft_entry__.build()
    assert "host module" in capsys.readouterr().err
