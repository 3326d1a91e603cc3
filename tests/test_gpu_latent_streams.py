"""The tensor-level calls on a stream that is not torch's current one, through `stream=`."""
import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref
from tests.test_gpu_latent_attention import Case

pytestmark = pytest.mark.gpu

KVS = [lib.KV_FP8_E4M3, lib.KV_BF16]
BUSY = 20_000_000                                       # cycles, some 10 ms


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("as_int", [False, True])
def test_workspace_is_not_handed_on(kv, as_int):
    """The current stream allocates and fills blocks of the workspace's size while the calls run."""
    c = Case([3000, 64, 0, 9000], 24, kv, seed=3)
    q, pool, table, lens = c.q.cuda(), c.pool.cuda(), c.table.cuda(), c.seqlens.cuda()
    s = torch.cuda.Stream()
    floats = lib.dsa_latent_attention_workspace()
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = torch.empty((c.R, c.H), device="cuda")
    torch.cuda.synchronize()
    outs, fills = [], []
    for _ in range(10):
        outs.append(lib.latent_attention(q[..., :512], q[..., 512:], pool, kv, table, lens, c.scale, lse=c.lse,
                                         dev_status=c.status, stream=s.cuda_stream if as_int else s))
        fills.append(torch.full((floats,), float("nan"), device="cuda"))
        fills.append(torch.full((c.R, c.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    for c.out in outs:
        c.check()


@pytest.mark.parametrize("kv", KVS)
def test_outputs_do_not_take_blocks_in_use(kv):
    """Blocks of the outputs' sizes, freed while the current stream has yet to write them."""
    c = Case([300, 70], 16, kv, seed=4)
    q, pool, table, lens = c.q.cuda(), c.pool.cuda(), c.table.cuda(), c.seqlens.cuda()
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = torch.empty((2, 16), device="cuda")
    cu = torch.tensor([0, 300, 370], dtype=torch.int32, device="cuda")
    x = torch.randn((5, 3, 128), device="cuda").to(torch.bfloat16)
    want, _ = lib.qk_norm_rope(x, None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    for shape in ((2, 16, 512), (370, 576), (5, 3, 128), (lib.dsa_latent_attention_workspace() * 2,)):
        torch.empty(shape, dtype=torch.bfloat16, device="cuda").fill_(7)       # freed before it is filled
    c.out = lib.latent_attention(q[..., :512], q[..., 512:], pool, kv, table, lens, c.scale, lse=c.lse,
                                 dev_status=c.status, stream=s)
    back = lib.latent_load(pool, kv, table, cu, 370, stream=s)
    turned, _ = lib.qk_norm_rope(x, None, stream=s)
    torch.cuda.synchronize()
    c.check()
    assert torch.equal(turned, want)
    tokens = []
    for r, n in enumerate(c.lens):
        t = torch.arange(n)
        tokens.append(ref.tokens(c.pool, kv, c.table[r].long()[t // 64], t % 64))
    assert torch.equal(back.double().cpu(), torch.cat(tokens))


def test_outputs_outlive_their_last_name():
    """An output read by the current stream and dropped is not given to the call's stream meanwhile."""
    s = torch.cuda.Stream()
    x = torch.randn((64, 8, 128), device="cuda").to(torch.bfloat16)
    minus = -x
    want, _ = lib.qk_norm_rope(x, None)
    torch.cuda.synchronize()
    y, _ = lib.qk_norm_rope(x, None, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(BUSY)
    kept = y.clone()                                    # read after the sleep
    del y
    z, _ = lib.qk_norm_rope(minus, None, stream=s)       # would overwrite it at once
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(z, -want)
