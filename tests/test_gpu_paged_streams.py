"""The calls on the paged cache on streams other than torch's current one, side by side, captured and
replayed, and with a wait that runs out."""
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests.test_gpu_block_select import Case as SelectCase
from tests.test_gpu_paged_attention import Case
from tests.test_gpu_timeout import _build_variant

pytestmark = pytest.mark.gpu

KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16")]
BUSY = 20_000_000                                       # cycles, some 10 ms
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def args_of(c):
    k, v, ks, vs = c.pools.cuda()
    return [c.q.cuda(), k, v, c.table.cuda(), c.seqlens.cuda(), c.scale], dict(k_scale=ks, v_scale=vs)


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("as_int", [False, True])
def test_workspace_is_not_handed_on(kv, dtype, as_int):
    """The current stream allocates and fills blocks of the workspace's size while the calls run."""
    c = Case([3000, 64, 0, 9000], 24, 3, 128, kv, dtype, seed=3)
    args, more = args_of(c)
    s = torch.cuda.Stream()
    floats = lib.dsa_paged_attention_workspace(24, 3, 128)
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = torch.empty((c.R, c.heads), device="cuda")
    torch.cuda.synchronize()
    outs, fills = [], []
    for _ in range(10):
        outs.append(lib.paged_attention(*args, **more, lse=c.lse, dev_status=c.status,
                                        stream=s.cuda_stream if as_int else s))
        fills.append(torch.full((floats,), float("nan"), device="cuda"))
        fills.append(torch.full(c.q.shape, float("nan"), dtype=c.dtype, device="cuda"))
    torch.cuda.synchronize()
    for c.out in outs:
        c.check()


def test_outputs_do_not_take_blocks_in_use():
    """Blocks of the outputs' sizes, freed while the current stream has yet to write them."""
    c, sel = Case([300, 70], 16, 2, 64, "bf16", "bf16", seed=4), SelectCase([3000, 700], 16, 2, 64, "bf16", seed=4)
    args, more = args_of(c)
    sel.run(5)
    given = [x.cuda() for x in (sel.q, sel.bounds, sel.unit, sel.table, sel.seqlens)]
    lengths, new = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([64, 3], [2, 1]))
    free, table = torch.tensor([8, 9], dtype=torch.int32, device="cuda"), torch.tensor([[4, -1], [5, -1]], dtype=torch.int32, device="cuda")
    c.status, c.lse = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.empty((2, 16), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for shape in ((2, 16, 64), (2, 2, 5, 2), (5, 2), (2, 2), (3, 2), (1, 2), (lib.dsa_paged_attention_workspace(16, 2, 64) * 2,)):
        torch.empty(shape, dtype=torch.bfloat16, device="cuda").fill_(7)       # freed before it is filled
    c.out = lib.paged_attention(*args, **more, lse=c.lse, dev_status=c.status, stream=s)
    blocks = lib.block_select(*given, 5, stream=s)
    slots, positions, seqlens, cu, used = lib.request_slots(lengths, new, free, table, 5, stream=s)
    torch.cuda.synchronize()
    c.check()
    assert torch.equal(blocks.cpu(), sel.out)
    assert slots.tolist() == [512, 513, 323, -1, -1] and positions.tolist() == [64, 65, 3, 0, 0]
    assert seqlens.tolist() == [66, 4] and cu.tolist() == [0, 2, 3] and used.tolist() == [1]


@pytest.mark.parametrize("kv,dtype", KINDS)
def test_calls_side_by_side(kv, dtype):
    """Three streams, a workspace each, shapes that share their kernels."""
    cases = [Case([5000, 100 * i, 2000], 8 * (i + 1), 2, 128, kv, dtype, seed=20 + i) for i in range(3)]
    given = [args_of(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for c in cases:
        c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        c.outs = [(torch.empty(c.q.shape, dtype=c.dtype, device="cuda"), torch.empty((c.R, c.heads), device="cuda")) for _ in range(8)]
        c.ws = torch.empty(lib.dsa_paged_attention_workspace(c.heads, 2, 128), device="cuda")
    torch.cuda.synchronize()
    for i in range(8):
        for c, (args, more), s in zip(cases, given, streams):
            lib.paged_attention(*args, **more, out=c.outs[i][0], lse=c.outs[i][1], workspace=c.ws, dev_status=c.status, stream=s)
    torch.cuda.synchronize()
    for c in cases:
        for out, lse in c.outs:
            assert torch.equal(out, c.outs[0][0]) and torch.equal(lse, c.outs[0][1])
        c.out, c.lse = c.outs[0]
        c.check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("listed,W", [(False, 40), (False, 100), (True, 40)])
def test_replay_with_other_lengths_tables_and_lists(kv, dtype, listed, W):
    """Two graphs that share a workspace, replayed in turn after their inputs change in place."""
    def blocks_of(seed):
        g = torch.Generator().manual_seed(seed)
        return torch.randint(-2, 20, (3, 2, 6), generator=g).to(torch.int32) if listed else None
    sets = [[Case(lens, 8, 2, 64, kv, dtype, seed=i, W=W, blocks=blocks_of(i)) for i, lens in enumerate(l)]
            for l in ([[1, 2500, 64], [900, 0, 1]], [[300, 300, 2000], [0, 0, 65]])]
    ws = torch.empty(lib.dsa_paged_attention_workspace(8, 2, 64), device="cuda")
    graphs = []
    for first, _ in sets:
        pages = 100
        k, v, ks, vs = first.pools.cuda()
        state = dict(q=first.q.cuda(), table=first.table.cuda(), lens=first.seqlens.cuda(), out=torch.empty_like(first.q, device="cuda"),
                     lse=torch.empty((3, 8), device="cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"),
                     blocks=None if first.blocks is None else first.blocks.cuda())
        for name, x in (("k", k), ("v", v)):
            raw = torch.zeros((pages, 2, 64, 64), dtype=torch.uint8 if kv == "fp8" else x.dtype, device="cuda")
            state[name] = raw.view(x.dtype).transpose(1, 2)
        state["ks"] = state["vs"] = None
        if kv == "fp8":
            state["ks"], state["vs"] = torch.zeros((pages, 2, 64), device="cuda"), torch.zeros((pages, 2, 64), device="cuda")

        def call(s=state):
            lib.paged_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], 64 ** -0.5, blocks=s["blocks"], k_scale=s["ks"],
                                v_scale=s["vs"], out=s["out"], lse=s["lse"], workspace=ws, dev_status=s["status"])
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        graphs.append((graph, state))
    raw = (lambda x: x.view(torch.uint8)) if kv == "fp8" else (lambda x: x)
    for turn in (0, 1, 0):
        for (graph, s), cases in zip(graphs, sets):
            c = cases[turn]
            k, v, ks, vs = c.pools.cuda()
            raw(s["k"])[:k.shape[0]].copy_(raw(k))
            raw(s["v"])[:k.shape[0]].copy_(raw(v))
            if ks is not None:
                s["ks"][:k.shape[0]].copy_(ks)
                s["vs"][:k.shape[0]].copy_(vs)
            s["q"].copy_(c.q), s["table"].copy_(c.table), s["lens"].copy_(c.seqlens)
            if listed:
                s["blocks"].copy_(c.blocks)
            graph.replay()
        torch.cuda.synchronize()
        for (graph, s), cases in zip(graphs, sets):
            c = cases[turn]
            c.out, c.lse, c.status = s["out"], s["lse"], s["status"]
            c.check()


def test_first_calls_of_a_process_are_captured(tmp_path):
    """No call needs one before its capture."""
    code = tmp_path / "first.py"
    code.write_text("""
import torch
import sparse_attention_paged_gb300 as lib
int32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
q = torch.ones((2, 8, 64), device="cuda").to(torch.bfloat16)
k = torch.ones((4, 2, 64, 64), device="cuda").to(torch.bfloat16).transpose(1, 2)
v = torch.ones((4, 2, 64, 64), device="cuda").to(torch.bfloat16).transpose(1, 2)
wide = torch.zeros((2, 300), dtype=torch.int32, device="cuda")
table, lengths, new, free = int32([[0, 1], [2, 3]]), int32([70, 100]), int32([1, 1]), int32([])
bounds, unit = torch.zeros((4, 2, 2, 64), dtype=torch.int8, device="cuda"), torch.zeros((4, 2), device="cuda")
ws = torch.empty(lib.dsa_paged_attention_workspace(8, 2, 64), device="cuda")
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    slots, _, lens, _, _ = lib.request_slots(lengths, new, free, table, 2)
    lib.kv_store(q[:, :2] * 3, q[:, 2:4] * 3, slots, k, v)
    lib.block_bounds(k, table, lengths, lens, 1, bounds, unit)
    blocks = lib.block_select(q, bounds, unit, table, lens, 1, first=0, last=1)
    out = lib.paged_attention(q, k, v, table, lens, 0.1, blocks=blocks, workspace=ws)
    all_ = lib.paged_attention(q, k, v, wide, lens, 0.1, workspace=ws)
graph.replay()
torch.cuda.synchronize()
assert slots.tolist() == [64 + 6, 192 + 36] and blocks.tolist() == [[[1], [1]], [[1], [1]]], (slots, blocks)
assert (bounds[1, :, 0] == 96).all() and (out >= 1).all() and (all_ == 1).all()
""")
    r = subprocess.run([sys.executable, str(code)], cwd=ROOT, capture_output=True, text=True, timeout=300,
                       env={**os.environ, "PYTHONPATH": ROOT})
    assert r.returncode == 0, r.stderr


@pytest.fixture(scope="module")
def variant(tmp_path_factory):
    """A test-only build whose producers leave the first page of every CTA undelivered, with waits of some 10 ms."""
    L = _build_variant(str(tmp_path_factory.mktemp("timeout")))
    from sparse_attention_paged_gb300 import _native
    L.dsa_paged_attention.restype = ctypes.c_int
    L.dsa_paged_attention.argtypes = _native.load().dsa_paged_attention.argtypes
    return L


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("lens,W", [([40], None), ([1000], None), ([1000], 300), ([300, 0, 700, 64], None), ([300, 0, 20000, 64], None)])
def test_wait_that_runs_out(variant, kv, dtype, lens, W):
    """NaN for every row that has tokens, zeros for the others, a status, and a context that goes on."""
    c = Case(lens, 12, 2, 128, kv, dtype, seed=31, W=W)
    k, v, ks, vs = c.pools.cuda()
    q, table, seqlens = c.q.cuda(), c.table.cuda(), c.seqlens.cuda()
    out = torch.full(c.q.shape, 3.0, dtype=c.dtype, device="cuda")
    lse = torch.full((c.R, 12), 3.0, device="cuda")
    ws = torch.empty(lib.dsa_paged_attention_workspace(12, 2, 128), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    address = lambda x: None if x is None else x.data_ptr()                       # noqa: E731
    kinds = {"bf16": lib.KV_BF16, "fp16": lib.KV_FP16, "fp8": lib.KV_FP8_E4M3}
    st = variant.dsa_paged_attention(
        q.data_ptr(), q.stride(0), q.stride(1), c.R, 12, 2, 128, lib.FP16 if dtype == "fp16" else lib.BF16, c.scale,
        k.data_ptr(), k.stride(0), k.stride(1), k.stride(2), v.data_ptr(), v.stride(0), v.stride(1), v.stride(2),
        address(ks), address(vs), k.shape[0], kinds[kv], 64, table.data_ptr(), table.stride(0), table.shape[1],
        seqlens.data_ptr(), None, 0, 0, 0, out.data_ptr(), out.stride(0), out.stride(1), lse.data_ptr(), ws.data_ptr(),
        ws.numel(), status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()                      # returns: the kernel did not hang
    assert int(status) == 5                       # DSA_ERR_TIMEOUT
    for r, n in enumerate(lens):
        if n:
            assert torch.isnan(out[r].float()).all() and torch.isnan(lse[r]).all()
        else:
            assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    c.run().check()                               # the product library, in the same context
