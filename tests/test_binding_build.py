"""The compiled marshalling module never outlives what it was made of."""
import sys
import types

import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def dsa():
    __graft_entry__.build()
    import sparse_attention_long_gb300 as dsa
    return dsa


@pytest.fixture
def old(monkeypatch, tmp_path):
    """A module of an earlier build, in place of the package's own."""
    from sparse_attention_long_gb300 import _build
    path = tmp_path / "_binding.so"
    path.write_bytes(b"old")
    monkeypatch.setattr(_build, "BINDING", str(path))
    return _build, path


def test_a_failed_compilation_leaves_no_module(old, capsys):
    build, path = old
    build._build_binding([sys.executable, "-c", "import sys; sys.exit('no such header')"])
    assert not path.exists() and "no such header" in capsys.readouterr().err


def test_without_a_compiler_a_stale_module_goes_and_a_present_one_stays(old, monkeypatch):
    build, path = old
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    import os
    os.utime(path, (2e9, 2e9))                     # newer than every source
    assert build._binding_job("/usr/local/cuda/bin/nvcc", False) is None and path.exists()
    os.utime(path, (1, 1))
    assert build._binding_job("/usr/local/cuda/bin/nvcc", False) is None and not path.exists()


def test_only_a_module_of_the_present_sources_is_loaded(dsa, monkeypatch):
    import torch

    from sparse_attention_long_gb300 import _build
    assert _build.binding_stamp("2.9") != _build.binding_stamp("2.11")
    bound = []
    for stamp in (None, "", "0123456789abcdef"):
        other = types.ModuleType("sparse_attention_long_gb300._binding")
        other.bind = lambda *a: bound.append(a)
        if stamp is not None:
            other.stamp = stamp
        monkeypatch.setitem(sys.modules, other.__name__, other)
        monkeypatch.setattr(dsa, "_binding", other, raising=False)
        assert isinstance(dsa._load_native(), dsa._Absent) and not bound
    other.stamp = _build.binding_stamp(torch.__version__)
    assert dsa._load_native() is other and len(bound) == 1
    assert dsa._Absent().cache_fork() == 1         # nothing done: the Python code makes the call


def test_the_module_carries_the_stamp(dsa):
    from sparse_attention_long_gb300 import _build
    import os
    import torch
    if not os.path.exists(_build.BINDING):
        pytest.skip("built without PyTorch's or Python's headers")
    assert dsa._native.stamp == _build.binding_stamp(torch.__version__)
