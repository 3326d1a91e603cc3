"""What is compiled for whom (no GPU, and nothing is compiled here)."""
import os
import shutil
import subprocess
import sys
import sysconfig
import types

import pytest
import torch

from sparse_attention_paged_gb300 import _native

pytestmark = pytest.mark.skipif(shutil.which(_native.NVCC) is None and not os.path.exists(_native.LIB_PATH),
                                reason="nvcc not available and library not built")


@pytest.fixture
def built():
    _native.load_calls()


@pytest.mark.parametrize("where,name,value", [
    (torch, "__version__", "9.9.9"), (torch.version, "git_version", "0" * 40),
    (sysconfig, "get_config_var", lambda name: ".cpython-399-other.so")])
def test_another_torch_or_python_has_its_own_module(built, monkeypatch, where, name, value):
    """A module that was compiled against another torch's tensors is not loaded."""
    assert not _native.calls_stale()
    here = _native.calls_path()
    monkeypatch.setattr(where, name, value)
    assert _native.calls_path() != here
    assert _native.calls_stale() and not _native.is_stale()


def test_c_library_needs_no_torch_headers(monkeypatch, tmp_path):
    """The library is built and loaded where the module of the tensor-level calls cannot be."""
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w"):
            pass
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    def no_headers(*a):
        raise RuntimeError("torch/csrc/autograd/python_variable.h: no such file")
    monkeypatch.setattr(_native, "BUILD", str(tmp_path))
    monkeypatch.setattr(_native, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(_native, "_lib", None)
    monkeypatch.setattr(_native, "_calls", None)
    monkeypatch.setattr(_native, "_compile_calls", no_headers)
    monkeypatch.setattr(_native.subprocess, "run", run)
    assert _native.is_stale()
    _native.build()
    assert not _native.is_stale() and ran and all(cmd[0] == _native.NVCC for cmd in ran)
    with pytest.raises(RuntimeError, match="python_variable"):
        _native.build_calls()


BUILDER = """
import os, subprocess, sys, time, types
sys.path.insert(0, sys.argv[2])
from sparse_attention_paged_gb300 import _native
_native.BUILD = sys.argv[1]
_native.LIB_PATH = os.path.join(sys.argv[1], "lib.so")
_native._sources = lambda: [os.path.join(_native.CSRC, "dsa_api.cu")]

def run(cmd, **kw):
    out = cmd[cmd.index("-o") + 1]
    with open(os.path.join(sys.argv[1], "ran"), "a") as f:
        f.write("x")
    with open(out, "w"):
        time.sleep(0.3)
    return types.SimpleNamespace(returncode=0, stdout="", stderr="")

_native.subprocess = types.SimpleNamespace(run=run)
_native.build()
assert not _native.is_stale()
"""


def test_processes_do_not_build_at_once(tmp_path):
    """Three that find the build missing: one compiles and links, the others wait and take its files."""
    args = [sys.executable, "-c", BUILDER, str(tmp_path), _native.ROOT]
    running = [subprocess.Popen(args) for _ in range(3)]
    assert [p.wait(timeout=60) for p in running] == [0, 0, 0]
    assert (tmp_path / "ran").read_text() == "xx"
