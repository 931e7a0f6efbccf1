"""What the build needs and leaves: the library with nvcc alone, where there is
no torch or its headers do not compile; the binding's native part under a name
of its own for each torch and Python."""
import ctypes
import importlib
import os
import shutil
import subprocess

import pytest

import fp8_quantised_paged_kv_gb300 as kvq

B = importlib.import_module("fp8_quantised_paged_kv_gb300.build")


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build in an empty folder, of one source file."""
    if shutil.which(B._nvcc()) is None:
        pytest.skip("no nvcc")
    monkeypatch.setattr(B, "BUILD", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libkvq.so"))
    monkeypatch.setattr(B, "sources", lambda: [os.path.join(B.CSRC, "kvq_probe.cu")])
    monkeypatch.delattr(B, "NATIVE", raising=False)
    return tmp_path


def _no_torch(monkeypatch):
    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", missing)
    monkeypatch.setitem(__import__("sys").modules, "torch", None)


def test_the_library_builds_without_torch(small, monkeypatch):
    _no_torch(monkeypatch)
    lib = B.build()
    assert lib == str(small / "libkvq.so")
    ctypes.CDLL(lib).kvq_read_probe
    assert [x for x in os.listdir(small) if "native" in x] == []


def test_the_library_is_in_place_where_the_binding_does_not_compile(small, monkeypatch):
    run = subprocess.run

    def no_gxx(cmd, **kw):
        if cmd[0] == "g++":
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        return run(cmd, **kw)
    monkeypatch.setattr(subprocess, "run", no_gxx)
    with pytest.raises(RuntimeError, match="no such header"):
        B.build()
    assert os.path.exists(small / "libkvq.so")
    os.remove(small / "libkvq.so")
    assert os.path.exists(B.build(native=False))            # the library alone


def test_the_native_part_is_named_after_its_torch_and_python(monkeypatch):
    import sysconfig

    import torch
    here = B.native_path()
    assert torch.__version__.split("+")[0] in here and sysconfig.get_config_var("SOABI") in here
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.1.0")
    other = B.native_path()
    assert other != here and not os.path.exists(other)
    monkeypatch.undo()
    assert B.build_native() == here and os.path.exists(here)
    assert kvq._load_native().__file__ == here


def test_a_torch_without_metadata_is_found(monkeypatch):
    import torch

    def missing(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", missing)
    assert B.torch_version() == torch.__version__
