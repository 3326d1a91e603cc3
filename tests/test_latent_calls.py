"""The tensor-level calls' host side (no GPU): where their allocations belong."""
import contextlib
import types

import pytest
import torch

import sparse_attention_paged_gb300 as lib


class Tensor:
    """A stand-in for a CUDA tensor: notes the stream that was current at its creation."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, streams):
        self.shape, self.streams = shape, streams
        self.made_on, self.users = streams[-1], []

    def new_empty(self, shape, dtype=None):
        return Tensor(shape, self.streams)

    def record_stream(self, stream):
        self.users.append(stream)

    def stride(self, i):
        return 1


@pytest.fixture
def calls(monkeypatch):
    """torch.cuda's streams and the compiled calls replaced; `made` holds what the calls were given."""
    streams, made = ["current"], []

    @contextlib.contextmanager
    def scope(stream):
        streams.append(stream)
        yield
        streams.pop()

    def call(*args):
        made.extend(a for a in args if isinstance(a, Tensor) and a is not given)
        return 0

    given = Tensor((2, 4, 512), streams)
    monkeypatch.setattr(torch.cuda, "stream", scope)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: streams[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda address, device=None: address)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: Tensor(a, streams))
    monkeypatch.setattr(lib, "_calls", types.SimpleNamespace(
        qk_norm_rope=call, latent_load=call, latent_attention=call))
    monkeypatch.setattr(lib, "dsa_latent_attention_workspace", lambda: 1000)
    monkeypatch.setattr(lib, "dsa_indexer_logits_decode", call)
    return given, made


SIDE = types.SimpleNamespace(cuda_stream=7)
STREAMS = [(SIDE, SIDE), (5, 5), (0, "default")]
CALLS = {
    "qk_norm_rope": lambda x, stream: lib.qk_norm_rope(x, x, stream=stream),
    "latent_load": lambda x, stream: lib.latent_load(x, lib.KV_BF16, x, x, 3, stream=stream),
    "latent_attention": lambda x, stream: lib.latent_attention(x, x, x, lib.KV_BF16, x, x, 0.1, stream=stream),
    "indexer_logits": lambda x, stream: lib.indexer_logits("decode", x, x, x, x, 0, 0, 0, x, 0, x, 2, stream=stream),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream,want", STREAMS)
def test_allocations_belong_to_the_given_stream(calls, name, stream, want):
    """Outputs and the workspace come from the stream that the kernels run on; outputs are marked as
    in use on the current one too."""
    x, made = calls
    back = CALLS[name](x, stream)
    back = back if isinstance(back, tuple) else (back,)
    assert made and all(t.made_on == want for t in made)
    assert all(t in made and t.users == ["current"] for t in back)
    assert len(made) == len(back) + (name == "latent_attention")


@pytest.mark.parametrize("name", list(CALLS))
def test_allocations_of_the_current_stream(calls, name):
    x, made = calls
    CALLS[name](x, None)
    assert made and all(t.made_on == "current" and not t.users for t in made)


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("sliced", [False, True])
def test_lists_without_entries_are_refused(rows, sliced):
    """An empty list is not "every position": it has no address, as no list has none."""
    ql, qr = torch.zeros((rows, 8, 512), dtype=torch.bfloat16), torch.zeros((rows, 8, 64), dtype=torch.bfloat16)
    pool, lens = torch.zeros((2, 41984), dtype=torch.uint8), torch.ones(rows, dtype=torch.int32)
    idx = torch.zeros((rows, 5), dtype=torch.int32)[:, :0] if sliced else torch.zeros((rows, 0), dtype=torch.int32)
    with pytest.raises(ValueError, match="at least one entry"):
        lib.latent_attention(ql, qr, pool, lib.KV_FP8_E4M3, torch.zeros((1, 2), dtype=torch.int32), lens, 0.1, idx=idx)
