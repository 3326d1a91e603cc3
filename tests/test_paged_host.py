"""Host-side argument checks of the calls on the paged cache of keys and values (no GPU: every call
here is refused, or has nothing to launch, before any device work)."""
import contextlib
import os
import shutil
import types

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from sparse_attention_paged_gb300 import _native
from tests import paged_ref as ref

pytestmark = pytest.mark.skipif(shutil.which(_native.NVCC) is None and
                                not os.path.exists(_native.LIB_PATH),
                                reason="nvcc not available and library not built")

A = 0x10000          # a fake, aligned device address
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
FP8, BF16, FP16 = lib.KV_FP8_E4M3, lib.KV_BF16, lib.KV_FP16


def slots(**kw):
    args = dict(lengths=A, new_tokens=A + 4096, n_req=3, free_pages=A, n_free=8, block_table=A, bt_stride=4, W=4,
                page_size=64, n=10, slots=A, positions=A, seqlens=A + 8192, cu_rows=A, used=A, stream=0)
    args.update(kw)
    return lib.dsa_request_slots(**args)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=0, n_req=0, cu_rows=None, used=None)),
    (INVALID, dict(n=-1)), (INVALID, dict(n_req=-1)), (INVALID, dict(n_free=-1)), (INVALID, dict(W=0)),
    (INVALID, dict(bt_stride=3)), (INVALID, dict(bt_stride=0)), (INVALID, dict(bt_stride=-4)),
    (INVALID, dict(lengths=None)), (INVALID, dict(new_tokens=None)), (INVALID, dict(block_table=None)),
    (INVALID, dict(slots=None)), (INVALID, dict(free_pages=None)), (INVALID, dict(seqlens=A)),
    (INVALID, dict(seqlens=A + 4096)),
    (UNSUPPORTED, dict(page_size=16)), (UNSUPPORTED, dict(W=2 ** 25, bt_stride=2 ** 25)),
    (MISALIGNED, dict(lengths=A + 2)), (MISALIGNED, dict(slots=A + 1)), (MISALIGNED, dict(block_table=A + 2)),
    (MISALIGNED, dict(used=A + 3)),
])
def test_slots_refusals(want, kw):
    assert slots(**kw) == want


def store(**kw):
    args = dict(k=A, k_token_stride=1024, k_head_stride=128, v=A, v_token_stride=1024, v_head_stride=128, n=4, Hkv=8,
                D=128, dtype=lib.BF16, slot_mapping=A, k_cache=A, kc_page_stride=65536, kc_slot_stride=1024,
                kc_head_stride=128, v_cache=A, vc_page_stride=65536, vc_slot_stride=128, vc_head_stride=8192,
                k_scale=A, v_scale=A, num_pages=5, kv_dtype=FP8, page_size=64, stream=0)
    args.update(kw)
    return lib.dsa_kv_store(**args)


POOL = [
    (INVALID, dict(k_cache=None)), (INVALID, dict(num_pages=0)), (INVALID, dict(kc_slot_stride=64)),
    (INVALID, dict(kc_head_stride=0)), (INVALID, dict(kc_page_stride=-65536)), (INVALID, dict(k_scale=None)),
    (INVALID, dict(kv_dtype=3)), (INVALID, dict(kv_dtype=-1)), (INVALID, dict(Hkv=0)), (INVALID, dict(Hkv=-2)),
    (UNSUPPORTED, dict(D=96)), (UNSUPPORTED, dict(D=256)), (UNSUPPORTED, dict(page_size=32)),
    (UNSUPPORTED, dict(num_pages=2 ** 25)),
    (MISALIGNED, dict(k_cache=A + 8)), (MISALIGNED, dict(kc_slot_stride=1032)), (MISALIGNED, dict(kc_head_stride=136)),
    (MISALIGNED, dict(kc_page_stride=65544)), (MISALIGNED, dict(k_scale=A + 4)),
]
VALUES = [
    (INVALID, dict(v_cache=None)), (INVALID, dict(v_scale=None)), (INVALID, dict(vc_head_stride=64)),
    (MISALIGNED, dict(v_cache=A + 4)), (MISALIGNED, dict(vc_slot_stride=136)), (MISALIGNED, dict(v_scale=A + 8)),
    (INVALID, dict(dtype=lib.FP32)), (UNSUPPORTED, dict(kv_dtype=FP16)),
    (UNSUPPORTED, dict(kv_dtype=BF16, dtype=lib.FP16)),
]


@pytest.mark.parametrize("want,kw", POOL + VALUES + [
    (OK, dict(n=0)), (OK, dict(n=0, k=None, v=None, slot_mapping=None)),
    (OK, dict(n=0, kv_dtype=BF16, k_scale=None, v_scale=None)),
    (OK, dict(n=0, num_pages=1, kc_page_stride=3)), (OK, dict(n=0, Hkv=1, kc_head_stride=0, vc_head_stride=5)),
    (INVALID, dict(n=-1)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(slot_mapping=None)),
    (UNSUPPORTED, dict(n=2 ** 30)),
    (MISALIGNED, dict(k=A + 8)), (MISALIGNED, dict(v_token_stride=1028)), (MISALIGNED, dict(k_head_stride=132)),
    (MISALIGNED, dict(slot_mapping=A + 2)),
])
def test_store_refusals(want, kw):
    assert store(**kw) == want


def bounds(**kw):
    args = dict(k_cache=A, kc_page_stride=65536, kc_slot_stride=1024, kc_head_stride=128, k_scale=A, num_pages=5,
                kv_dtype=FP8, Hkv=8, D=128, page_size=64, block_table=A, bt_stride=4, W=4, starts=A, seqlens=A,
                n_req=3, max_tokens=70, bounds=A, bound_scale=A, stream=0)
    args.update(kw)
    return lib.dsa_block_bounds(**args)


@pytest.mark.parametrize("want,kw", POOL + [
    (OK, dict(n_req=0)), (OK, dict(max_tokens=0)), (OK, dict(n_req=0, seqlens=None, bounds=None, bound_scale=None)),
    (INVALID, dict(n_req=-1)), (INVALID, dict(max_tokens=-1)), (INVALID, dict(W=0)), (INVALID, dict(bt_stride=3)),
    (INVALID, dict(seqlens=None)), (INVALID, dict(bounds=None)), (INVALID, dict(bound_scale=None)),
    (INVALID, dict(block_table=None)), (UNSUPPORTED, dict(n_req=2 ** 30)),
    (MISALIGNED, dict(bounds=A + 8)), (MISALIGNED, dict(bound_scale=A + 2)), (MISALIGNED, dict(starts=A + 1)),
])
def test_bounds_refusals(want, kw):
    assert bounds(**kw) == want


def select(**kw):
    args = dict(q=A, q_row_stride=4096, q_head_stride=128, rows=2, Hq=32, Hkv=8, D=128, dtype=lib.BF16, bounds=A,
                bound_scale=A, num_pages=5, block_table=A, bt_stride=4, W=4, page_size=64, seqlens=A, k=3, first=1,
                last=1, blocks=A, stream=0)
    args.update(kw)
    return lib.dsa_block_select(**args)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(rows=0)), (OK, dict(rows=0, q=None, bounds=None, blocks=None, seqlens=None)),
    (INVALID, dict(rows=-1)), (INVALID, dict(Hq=0)), (INVALID, dict(Hq=30)), (INVALID, dict(Hkv=0)),
    (INVALID, dict(dtype=2)), (INVALID, dict(k=0)), (INVALID, dict(first=-1)), (INVALID, dict(last=-1)),
    (INVALID, dict(first=2, last=2)), (INVALID, dict(first=2 ** 31 - 1, last=2 ** 31 - 1)),
    (INVALID, dict(num_pages=0)), (INVALID, dict(q=None)), (INVALID, dict(bounds=None)),
    (INVALID, dict(bound_scale=None)), (INVALID, dict(seqlens=None)), (INVALID, dict(blocks=None)),
    (INVALID, dict(W=0)), (INVALID, dict(bt_stride=2)),
    (UNSUPPORTED, dict(D=32)), (UNSUPPORTED, dict(page_size=128)), (UNSUPPORTED, dict(W=32769, bt_stride=32769)),
    (UNSUPPORTED, dict(Hq=1025 * 8)), (UNSUPPORTED, dict(rows=2 ** 29)),
    (MISALIGNED, dict(q=A + 8)), (MISALIGNED, dict(q_row_stride=4100)), (MISALIGNED, dict(bounds=A + 4)),
    (MISALIGNED, dict(bound_scale=A + 2)), (MISALIGNED, dict(blocks=A + 2)),
])
def test_select_refusals(want, kw):
    assert select(**kw) == want


def attention(**kw):
    args = dict(q=A, q_row_stride=4096, q_head_stride=128, rows=2, Hq=32, Hkv=8, D=128, dtype=lib.BF16, scale=0.1,
                k_cache=A, kc_page_stride=65536, kc_slot_stride=1024, kc_head_stride=128, v_cache=A,
                vc_page_stride=65536, vc_slot_stride=128, vc_head_stride=8192, k_scale=A, v_scale=A, num_pages=5,
                kv_dtype=FP8, page_size=64, block_table=A, bt_stride=4, W=4, seqlens=A, blocks=None,
                blocks_row_stride=0, blocks_head_stride=0, k=0, out=A, out_row_stride=4096, out_head_stride=128,
                lse=None, workspace=A, workspace_floats=2 ** 40, stream=0)
    args.update(kw)
    return lib.dsa_paged_attention(**args)


@pytest.mark.parametrize("want,kw", POOL + VALUES + [
    (OK, dict(rows=0)), (OK, dict(rows=0, q=None, out=None, workspace=None, seqlens=None, block_table=None)),
    (INVALID, dict(rows=-1)), (INVALID, dict(Hq=0)), (INVALID, dict(Hq=33)), (INVALID, dict(scale=float("inf"))),
    (INVALID, dict(scale=float("nan"))), (INVALID, dict(blocks=A, k=0)), (INVALID, dict(blocks=A, k=2, blocks_row_stride=-1)),
    (INVALID, dict(blocks=A, k=2, blocks_head_stride=-8)), (INVALID, dict(q=None)), (INVALID, dict(out=None)),
    (INVALID, dict(workspace=None)), (INVALID, dict(seqlens=None)), (INVALID, dict(block_table=None)),
    (INVALID, dict(W=0)), (INVALID, dict(bt_stride=3)),
    (UNSUPPORTED, dict(W=2 ** 25, bt_stride=2 ** 25)), (UNSUPPORTED, dict(rows=2 ** 27)),
    (UNSUPPORTED, dict(blocks=A, k=2 ** 28)),
    (MISALIGNED, dict(q=A + 8)), (MISALIGNED, dict(q_head_stride=132)), (MISALIGNED, dict(out=A + 2)),
    (MISALIGNED, dict(out_row_stride=4100)), (MISALIGNED, dict(workspace=A + 4)), (MISALIGNED, dict(lse=A + 2)),
    (MISALIGNED, dict(blocks=A + 2, k=2)),
])
def test_attention_refusals(want, kw):
    assert attention(**kw) == want


def test_workspace_of_shapes_that_are_not_taken():
    for shape in ((0, 1, 64), (8, 0, 64), (8, 3, 64), (8, 2, 96)):
        assert lib.dsa_paged_attention_workspace(*shape) == -1


# ---- the tensor level ---------------------------------------------------------------

def tensors(kv=torch.bfloat16, dtype=torch.bfloat16, rows=2, heads=8, kv_heads=2, dim=64, pages=3):
    int32 = dict(dtype=torch.int32)
    cache = torch.zeros((pages, 64, kv_heads, dim), dtype=torch.uint8 if kv == torch.float8_e4m3fn else kv)
    cache = cache.view(kv)
    scale = torch.ones((pages, kv_heads, 64)) if kv == torch.float8_e4m3fn else None
    return dict(q=torch.zeros((rows, heads, dim), dtype=dtype), k_cache=cache, v_cache=cache.clone(),
                block_table=torch.zeros((rows, 3), **int32), seqlens=torch.ones(rows, **int32), scale=0.1,
                k_scale=scale, v_scale=scale, workspace=torch.zeros(10))


E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("match,change", [
    ("q: ", dict(q=torch.zeros((2, 8, 64)))), ("q: ", dict(q=torch.zeros((2, 64), dtype=torch.bfloat16))),
    ("q: ", dict(q=torch.zeros((2, 8, 128), dtype=torch.bfloat16)[..., ::2])),
    ("k_cache: ", dict(k_cache=torch.zeros((3, 32, 2, 64), dtype=torch.bfloat16))),
    ("k_cache: ", dict(k_cache=torch.zeros((3, 64, 2, 64)))),
    ("k_cache: ", dict(q=torch.zeros((2, 8, 128), dtype=torch.bfloat16))),
    ("v_cache: ", dict(v_cache=torch.zeros((3, 64, 2, 64), dtype=torch.float16))),
    ("v_cache: ", dict(v_cache=torch.zeros((2, 64, 2, 64), dtype=torch.bfloat16))),
    ("seqlens: ", dict(seqlens=torch.ones(3, dtype=torch.int32))), ("seqlens: ", dict(seqlens=None)),
    ("seqlens: ", dict(seqlens=torch.ones(2, dtype=torch.int64))),
    ("block_table: ", dict(block_table=torch.zeros((3, 3), dtype=torch.int32))),
    ("blocks: ", dict(blocks=torch.zeros((2, 3, 4), dtype=torch.int32))),
    ("blocks: ", dict(blocks=torch.zeros((2, 4), dtype=torch.int32))),
    ("at least one entry", dict(blocks=torch.zeros((2, 2, 0), dtype=torch.int32))),
    ("k_scale", dict(k_scale=torch.ones((3, 2, 64)))), ("out: ", dict(out=torch.zeros((2, 8, 64), dtype=torch.float16))),
    ("lse: ", dict(lse=torch.zeros((2, 4)))), ("workspace: ", dict(workspace=torch.zeros(10, dtype=torch.float64))),
    ("CUDA tensor", dict()),
])
def test_attention_tensors(match, change):
    args = {**tensors(), **change}
    args.setdefault("out", torch.zeros((2, 8, 64), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match=match):
        lib.paged_attention(**args)


@pytest.mark.parametrize("scale", [None, torch.ones((3, 64, 2)), torch.ones((3, 2, 64), dtype=torch.float64)])
def test_fp8_caches_need_their_scales(scale):
    args = {**tensors(E4M3), "v_scale": scale, "out": torch.zeros((2, 8, 64), dtype=torch.bfloat16)}
    with pytest.raises(ValueError, match="v_scale: "):
        lib.paged_attention(**args)
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="v_scale: "):
        lib.kv_store(k, k, torch.zeros(4, dtype=torch.int32), args["k_cache"], args["v_cache"],
                     k_scale=args["k_scale"], v_scale=scale)


@pytest.mark.parametrize("match,change", [
    ("v: ", dict(v=torch.zeros((4, 2, 64), dtype=torch.float16))), ("v: ", dict(v=torch.zeros((3, 2, 64), dtype=torch.bfloat16))),
    ("k: ", dict(k=torch.zeros((4, 128), dtype=torch.bfloat16))),
    ("v_cache: ", dict(k_cache=torch.zeros((3, 64, 1, 64), dtype=torch.bfloat16))),
    ("slot_mapping: ", dict(slot_mapping=torch.zeros(5, dtype=torch.int32))), ("slot_mapping: ", dict(slot_mapping=None)),
    ("CUDA tensor", dict()),
])
def test_store_tensors(match, change):
    k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    cache = torch.zeros((3, 64, 2, 64), dtype=torch.bfloat16)
    args = {**dict(k=k, v=k, slot_mapping=torch.zeros(4, dtype=torch.int32), k_cache=cache, v_cache=cache.clone()), **change}
    with pytest.raises(ValueError, match=match):
        lib.kv_store(**args)


@pytest.mark.parametrize("match,change", [
    ("bounds: ", dict(bounds=torch.zeros((3, 2, 2, 64)))), ("bounds: ", dict(bounds=torch.zeros((3, 2, 2, 128), dtype=torch.int8))),
    ("bound_scale: ", dict(bound_scale=torch.zeros((3, 1)))), ("bound_scale: ", dict(bound_scale=None)),
    ("CUDA tensor", dict()),
])
def test_box_tensors(match, change):
    t = tensors()
    args = {**dict(bounds=torch.zeros((3, 2, 2, 64), dtype=torch.int8), bound_scale=torch.zeros((3, 2))), **change}
    with pytest.raises(ValueError, match=match):
        lib.block_bounds(t["k_cache"], t["block_table"], None, t["seqlens"], 5, args["bounds"], args["bound_scale"])
    with pytest.raises(ValueError, match=match):
        lib.block_select(t["q"], args["bounds"], args["bound_scale"], t["block_table"], t["seqlens"], 2,
                         out=torch.zeros((2, 2, 2), dtype=torch.int32))


@pytest.mark.parametrize("match,change", [
    ("lengths: ", dict(lengths=torch.zeros((2, 1), dtype=torch.int32))), ("new_tokens: ", dict(new_tokens=torch.zeros(3, dtype=torch.int32))),
    ("free_pages", dict(free_pages=None)), ("block_table: ", dict(block_table=torch.zeros((1, 4), dtype=torch.int32))),
    ("block_table: ", dict(block_table=torch.zeros(4, dtype=torch.int32))), ("slots: ", dict(slots=torch.zeros(3, dtype=torch.int32))),
    ("cu_rows: ", dict(cu_rows=torch.zeros(2, dtype=torch.int32))), ("CUDA tensor", dict()),
])
def test_slots_tensors(match, change):
    two = torch.zeros(2, dtype=torch.int32)
    args = {**dict(lengths=two, new_tokens=two.clone(), free_pages=torch.zeros(4, dtype=torch.int32),
                   block_table=torch.zeros((2, 4), dtype=torch.int32), n=5), **change}
    with pytest.raises(ValueError, match=match):
        lib.request_slots(**args)


# ---- where allocations belong ---------------------------------------------------------

class Tensor:
    """A stand-in for a CUDA tensor: notes the stream that was current at its creation."""
    is_cuda, device = True, "cuda:0"

    def __init__(self, shape, streams):
        self.shape, self.streams, self.made_on, self.users = shape, streams, streams[-1], []

    def new_empty(self, shape, dtype=None):
        return Tensor(shape, self.streams)

    def record_stream(self, stream):
        self.users.append(stream)


CALLS = {
    "request_slots": (lambda x, stream: lib.request_slots(x, x, x, x, 4, stream=stream), 5, 5),
    "block_select": (lambda x, stream: lib.block_select(x, x, x, x, x, 3, stream=stream), 1, 1),
    "paged_attention": (lambda x, stream: lib.paged_attention(x, x, x, x, x, 0.1, stream=stream), 1, 2),
}


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("stream,want", [(types.SimpleNamespace(cuda_stream=7), None), (5, 5), (0, "default"), (None, "current")])
def test_allocations_belong_to_the_given_stream(monkeypatch, name, stream, want):
    streams, made = ["current"], []

    @contextlib.contextmanager
    def scope(s):
        streams.append(s)
        yield
        streams.pop()

    given = Tensor((2, 4, 64), streams)

    def call(*args):
        made.extend(a for a in args if isinstance(a, Tensor) and a is not given)
        return 0
    monkeypatch.setattr(torch.cuda, "stream", scope)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: streams[-1])
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda address, device=None: address)
    monkeypatch.setattr(lib, "_calls", types.SimpleNamespace(request_slots=call, block_select=call, paged_attention=call))
    monkeypatch.setattr(lib, "dsa_paged_attention_workspace", lambda *shape: 1000)
    run, returned, allocated = CALLS[name]
    back = run(given, stream)
    back = back if isinstance(back, tuple) else (back,)
    want = stream if stream is not None and want is None else want
    assert len(back) == returned and len(made) == allocated
    assert all(t.made_on == want for t in made)
    assert all(t.users == ([] if stream is None else ["current"]) for t in back)


# ---- the references themselves ----------------------------------------------------------

def test_reference_scales_and_boxes():
    assert ref.scale_of(0.0) == 2.0 ** -126 and ref.scale_of(448.0) == 1.0 and ref.scale_of(448.1) == 2.0
    assert ref.scale_of(127.0, 127.0) == 1.0 and ref.scale_of(127.1, 127.0) == 2.0 and ref.scale_of(2.0 ** -140) == 2.0 ** -126
    g = torch.Generator().manual_seed(1)
    keys = torch.randn((50, 64), generator=g).double()
    codes, unit = ref.box(keys)
    assert ((keys <= codes[0].double() * unit) & (keys >= codes[1].double() * unit)).all()
    assert codes.abs().max() > 63


def test_reference_score_bounds_every_key():
    """The choice's score is at least the group's summed products with any key of the page (one factor for all)."""
    g = torch.Generator().manual_seed(2)
    q, keys = torch.randn((4, 64), generator=g).double(), torch.randn((12, 64, 64), generator=g).double()
    boxes = torch.stack([ref.box(k)[0] for k in keys])
    unit = torch.tensor([ref.box(k)[1] for k in keys])
    x = 2.0 ** (20 - torch.frexp(q.abs().max())[1].item())
    whole = torch.round(q * x)
    above, below = whole.clamp(min=0).sum(0), (-whole).clamp(min=0).sum(0)
    s = 0
    while max(above.max(), below.max()) > 127 * 2 ** s:
        s += 1
    p, m = torch.ceil(above / 2 ** s), torch.ceil(below / 2 ** s)
    score = (boxes[:, 0].double() @ p - boxes[:, 1].double() @ m) * unit.double() * 2 ** s / x
    best = (keys @ q.T).sum(-1).amax(-1)
    assert (score >= best - 1e-4).all()
