"""Forms of latent attention's arguments: one table for all rows without lists, lists with more heads
than one group, prompts of several requests, lists inside wider rows; and the same bits every time."""
import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests.test_gpu_latent_attention import Case

pytestmark = pytest.mark.gpu

KVS = [lib.KV_FP8_E4M3, lib.KV_BF16]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("H", [16, 64, 100])
@pytest.mark.parametrize("form", ["row", "one row", "expanded"])
def test_prompt_over_a_shared_table_without_lists(kv, H, form):
    """Every query token of a prompt attends to all positions up to its own."""
    n, ctx = 150, 500
    c = Case([ctx - n + 1 + i for i in range(n)], H, kv, shared=True, seed=H)
    row = c.table.cuda()
    table = {"row": row, "one row": row[None], "expanded": row[None].expand(n, -1)}[form]
    q = c.q.cuda()
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = torch.empty((n, H), device="cuda")
    c.out = lib.latent_attention(q[..., :512], q[..., 512:], c.pool.cuda(), kv, table, c.seqlens.cuda(),
                                 c.scale, lse=c.lse, dev_status=c.status)
    torch.cuda.synchronize()
    c.check(rows=list(range(0, n, 11)) + [n - 1])


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("H", [65, 100, 128])
def test_lists_with_more_heads_than_a_group(kv, H):
    Case([0, 1, 40, 64, 65, 500, 1000, 2500], H, kv, k=190, seed=H).run().check()


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("k", [0, 100])
def test_prompts_of_several_requests(kv, k):
    """The block table holds a request's row once for each of its query tokens."""
    counts, contexts = [40, 1, 90], [300, 70, 129]
    lens = [ctx - n + 1 + i for n, ctx in zip(counts, contexts) for i in range(n)]
    c = Case(lens, 24, kv, k=k, seed=21)
    W = c.table.shape[1]
    rows = torch.full((3, W), 2 ** 31 - 1, dtype=torch.int32)
    perm = torch.randperm(len(c.pool), generator=torch.Generator().manual_seed(3)).to(torch.int32)
    at = 0
    for r, ctx in enumerate(contexts):
        m = (ctx + 63) // 64
        rows[r, :m] = perm[at:at + m]
        at += m
    c.table = rows.repeat_interleave(torch.tensor(counts), dim=0)
    c.run().check(rows=list(range(0, len(lens), 7)) + [39, 40, 41])


@pytest.mark.parametrize("kv", KVS)
def test_lists_inside_wider_rows(kv):
    """The first entries of longer lists, through their stride."""
    c = Case([300, 5, 700, 64], 16, kv, k=130, seed=22)
    wide = torch.full((4, 200), 3, dtype=torch.int32)
    wide[:, :130] = c.idx
    q, lists = c.q.cuda(), wide.cuda()
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = torch.empty((4, 16), device="cuda")
    c.out = lib.latent_attention(q[..., :512], q[..., 512:], c.pool.cuda(), kv, c.table.cuda(), c.seqlens.cuda(),
                                 c.scale, idx=lists[:, :130], lse=c.lse, dev_status=c.status)
    torch.cuda.synchronize()
    c.check()


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("lens,H,k", [([4096], 16, 512), ([4096, 9000, 300, 7] * 8, 64, 700), ([30000], 128, 0),
                                      ([900] * 180, 37, 0)])
def test_the_same_bits_every_time(kv, lens, H, k):
    """No result depends on the order in which CTAs finish, nor on what the workspace held."""
    c = Case(lens, H, kv, k=k, seed=23)
    first, lse = None, None
    for i in range(5):
        work = torch.full((lib.dsa_latent_attention_workspace(),), float("nan") if i % 2 else 3e38, device="cuda")
        c.run(workspace=work)
        assert int(c.status) == 0
        if first is None:
            first, lse = c.out, c.lse
        assert torch.equal(c.out, first) and torch.equal(c.lse, lse)
