"""What is compiled for whom (no GPU, and nothing is compiled here)."""
import os
import shutil
import sysconfig

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
    assert not _native.is_stale()
    here = _native.calls_path()
    monkeypatch.setattr(where, name, value)
    assert _native.calls_path() != here
    assert _native.is_stale()
