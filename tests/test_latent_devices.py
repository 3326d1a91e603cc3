"""Tensors of another CUDA device are refused before any device work (fake tensors: their device is
a name, so no second GPU is needed)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_attention_paged_gb300 as lib


def calls(devices):
    """Each tensor-level call's tensors, one device after another from `devices`."""
    def t(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=next(devices))

    def ints(*shape):
        return t(*shape, dtype=torch.int32)

    def pool():
        return t(2, 41984, dtype=torch.uint8)
    return {
        "qk_norm_rope": lambda: lib.qk_norm_rope(t(3, 4, 128), t(3, 1, 128)),
        "latent_store": lambda: lib.latent_store(t(3, 512), t(3, 64), ints(3), pool(), lib.KV_FP8_E4M3),
        "latent_load": lambda: lib.latent_load(pool(), lib.KV_FP8_E4M3, ints(1, 2), ints(2), 5),
        "latent_attention": lambda: lib.latent_attention(t(3, 8, 512), t(3, 8, 64), pool(), lib.KV_FP8_E4M3,
                                                         ints(1, 2), ints(3), 0.1),
    }


@pytest.fixture(autouse=True)
def only_names(monkeypatch):
    """A fake tensor's first use would otherwise make a real one on its device."""
    monkeypatch.setattr(torch.cuda, "is_available", lambda: False)


NAMES = ["qk_norm_rope", "latent_store", "latent_load", "latent_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_two_devices_in_one_call(name):
    with FakeTensorMode():
        with pytest.raises(ValueError, match="more than one CUDA device"):
            calls(iter(["cuda:0"] + ["cuda:1"] * 9))[name]()


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_another_device_than_the_current_one(name):
    assert torch.cuda.current_device() == 0
    with FakeTensorMode():
        with pytest.raises(ValueError, match="not on the current CUDA device"):
            calls(iter(["cuda:1"] * 10))[name]()
