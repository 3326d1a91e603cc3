"""Attention over the latent cache on the GPU against a 64-bit reference."""
import math

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

KVS = [lib.KV_FP8_E4M3, lib.KV_BF16]


class Case:
    """Inputs of one call on the CPU, its run on the GPU and the check of its rows."""

    def __init__(self, lens, H, kv, k=0, seed=0, shared=False, W=None, scale=192 ** -0.5, gap=0, q_size=1.0):
        g = torch.Generator().manual_seed(seed)
        R = len(lens)
        self.R, self.H, self.kv, self.scale, self.lens = R, H, kv, scale, lens
        W = W or max(1, max((max(n, 0) + 63) // 64 for n in lens))
        used = W if shared else sum((max(min(n, W * 64), 0) + 63) // 64 for n in lens)
        self.pool = ref.random_pool(used + 1, kv, g, ref.PAGE_BYTES[kv] + gap)
        perm = torch.randperm(used + 1, generator=g).to(torch.int32)
        if shared:
            self.table = perm[:W].clone()
        else:
            self.table = torch.full((R, W), 2 ** 31 - 1, dtype=torch.int32)   # never a page
            at = 0
            for r, n in enumerate(lens):
                m = (max(min(n, W * 64), 0) + 63) // 64
                self.table[r, :m] = perm[at:at + m]
                at += m
        self.seqlens = torch.tensor(lens, dtype=torch.int32)
        self.idx = None
        if k:
            self.idx = torch.full((R, k), -1, dtype=torch.int32)
            for r, n in enumerate(lens):
                m = min(k, max(n, 0))
                self.idx[r, :m] = torch.randperm(max(n, 1), generator=g)[:m].sort().values.to(torch.int32)
        self.q = (q_size * torch.randn((R, H, 576), generator=g)).to(torch.bfloat16)

    def run(self, lse=True, workspace=None, out=None):
        q = self.q.cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lse = torch.full((self.R, self.H), 5.0, device="cuda") if lse else None
        self.out = lib.latent_attention(
            q[..., :512], q[..., 512:], self.pool.cuda(), self.kv, self.table.cuda(),
            self.seqlens.cuda(), self.scale, idx=None if self.idx is None else self.idx.cuda(),
            out=out, lse=self.lse, workspace=workspace, dev_status=self.status)
        torch.cuda.synchronize()
        return self

    def check(self, rows=None, status=0):
        assert int(self.status) == status
        out = self.out.double().cpu()
        for r in range(self.R) if rows is None else rows:
            t = torch.tensor(ref.visible(r, self.seqlens, self.idx), dtype=torch.long)
            row = self.table if self.table.dim() == 1 else self.table[r]
            kv = ref.tokens(self.pool, self.kv, row.long()[t // 64], t % 64)
            want, lse, bound, lse_bound = ref.attention_row(self.q[r].double(), kv, self.scale)
            assert torch.isfinite(out[r]).all(), r
            d = (out[r] - want).abs()
            assert (d <= bound).all(), (r, float((d - bound).max()), float(d.max()))
            if self.lse is None:
                continue
            got = self.lse[r].double().cpu()
            if not len(t):
                assert (got == -math.inf).all()
            else:
                assert ((got - lse).abs() <= lse_bound).all(), (r, float((got - lse).abs().max()))
        return self


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 128, 200])
def test_one_row(kv, n):
    Case([n], 64, kv, seed=n).run().check()


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("H", [1, 7, 16, 37, 64, 65, 100, 128])
def test_head_counts(kv, H):
    Case([130, 1, 0, 300], H, kv, seed=H).run().check()


@pytest.mark.parametrize("kv", KVS)
def test_lengths_of_every_kind(kv):
    """Empty, negative, short and long rows: many rows per slice, rows cut by slices."""
    lens = [0, 5, -3, 64, 1, 0, 0, 4097, 63, 65, 129, 0, 2000] + [17] * 40 + [0] * 5 + [700, 0]
    Case(lens, 64, kv, seed=2, gap=256).run().check()


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("k", [1, 63, 64, 65, 300])
def test_selection_lists(kv, k):
    Case([0, 1, 40, 64, 65, 500, 1000, 2500], 64, kv, k=k, seed=k).run().check()


@pytest.mark.parametrize("kv", KVS)
def test_list_entries_that_do_not_count(kv):
    """Entries of -1 and at or past the length inside the list, repeats, any order."""
    c = Case([300, 300, 300, 300], 16, kv, k=130, seed=4)
    g = torch.Generator().manual_seed(44)
    c.idx[0] = torch.randint(-40, 400, (130,), generator=g, dtype=torch.int32)
    c.idx[1] = -1
    c.idx[2] = 17
    c.idx[3, :64] = -1                                    # a whole tile masked, then tokens
    c.run().check()


@pytest.mark.parametrize("kv", KVS)
def test_no_row_sees_anything(kv):
    c = Case([0, 0, -1], 24, kv, seed=1, W=2).run().check()
    assert (c.out == 0).all()


@pytest.mark.parametrize("kv", KVS)
def test_long_row_over_all_slices(kv):
    Case([30000], 8, kv, seed=6).run().check()
    Case([9000, 20000], 128, kv, seed=7).run().check()


@pytest.mark.parametrize("kv", KVS)
def test_prefill_shared_table(kv):
    n, ctx = 300, 900
    c = Case([ctx - n + 1 + i for i in range(n)], 64, kv, k=200, shared=True, seed=8).run()
    c.check(rows=list(range(0, n, 7)) + [n - 1])


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("scale", [192 ** -0.5, 2.0, -0.1, 0.0])
def test_scales(kv, scale):
    """Large scores move the running maximum again and again; zero weighs all alike."""
    Case([1000, 64], 20, kv, seed=9, scale=scale).run().check()


@pytest.mark.parametrize("kv", KVS)
def test_growing_scores_rescale(kv):
    """Scores that grow from tile to tile by more than the kept maximum's slack, and fall again."""
    c = Case([640], 8, kv, seed=10)
    latent, rope, scale = ref.page_views(c.pool, kv)
    t = torch.arange(640)
    # the rotated part carries the growth along q's direction
    direction = torch.ones(64)
    c.q[0, :, 512:] = direction.to(torch.bfloat16)
    grow = torch.cat([torch.linspace(0, 60, 320), torch.linspace(60, 0, 320)])
    page, slot = c.table[0].long()[t // 64], t % 64
    value = (grow[:, None] / (64 * c.scale) * direction).to(torch.bfloat16)
    if kv == lib.KV_BF16:
        v = c.pool[:, :73728].view(torch.bfloat16).view(-1, 64, 576).clone()
        v[page, slot, 512:] = value
        c.pool[:, :73728] = v.view(torch.uint8).view(v.shape[0], -1)
    else:
        v = c.pool[:, 32768:40960].clone().view(torch.bfloat16).view(-1, 64, 64)
        v[page, slot] = value
        c.pool[:, 32768:40960] = v.view(torch.uint8).view(v.shape[0], -1)
    c.run().check()


@pytest.mark.parametrize("kv", KVS)
def test_masked_places_hold_nan(kv):
    """Slots past the length, unselected tokens and unused pages are NaN: never read."""
    c = Case([70, 10], 16, kv, k=20, seed=11)
    keep = torch.zeros((c.pool.shape[0], 64), dtype=torch.bool)
    for r in range(2):
        t = torch.tensor(ref.visible(r, c.seqlens, c.idx))
        keep[c.table[r].long()[t // 64], t % 64] = True
    at = torch.nonzero(~keep)
    for part, size in (((0, 1152),) if kv == lib.KV_BF16 else ((0, 512), (32768, 128), (40960, 16))):
        for page, slot in at.tolist():
            c.pool[page, part + slot * size:part + (slot + 1) * size] = 0xff
    c.run().check()


@pytest.mark.parametrize("kv", KVS)
def test_nan_in_a_visible_token_stays_in_its_row(kv):
    c = Case([100, 100], 8, kv, seed=12)
    p = int(c.table[0, 1])
    if kv == lib.KV_BF16:
        c.pool[p, 3 * 1152:3 * 1152 + 2] = 0xff
    else:
        c.pool[p, 3 * 512] = 0x7f
    c.run()
    assert torch.isnan(c.out[0].float()).all()
    c.check(rows=[1])


@pytest.mark.parametrize("kv", KVS)
def test_bad_pages_and_lengths(kv):
    c = Case([100, 200, 64, 300], 64, kv, seed=13)
    c.table[1, 1] = c.pool.shape[0]
    c.table[2, 0] = -5
    c.run()
    assert torch.isnan(c.out[1:3].float()).all() and torch.isnan(c.lse[1:3]).all()
    c.check(rows=[0, 3], status=6)
    c = Case([100, 65, 3], 64, kv, seed=14, W=1)
    c.run()
    assert torch.isnan(c.out[:2].float()).all() and torch.isnan(c.lse[:2]).all()
    c.check(rows=[2], status=7)


@pytest.mark.parametrize("kv", KVS)
def test_bad_page_in_a_split_row(kv):
    c = Case([20000, 50], 16, kv, seed=15)
    c.table[0, 200] = 2 ** 30
    c.run()
    assert torch.isnan(c.out[0].float()).all()
    c.check(rows=[1], status=6)


@pytest.mark.parametrize("kv", KVS)
def test_strides_stream_and_no_lse(kv):
    """Queries as slices of a wider tensor, output heads-major, another stream, dirty workspace."""
    c = Case([500, 3, 129], 24, kv, seed=16)
    g = torch.Generator().manual_seed(1)
    wide = torch.full((3, 24, 640), float("nan"), dtype=torch.bfloat16)
    wide[..., 32:608] = c.q
    out = torch.full((24, 3, 520), 3.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((lib.dsa_latent_attention_workspace(),), float("nan"), device="cuda")
    s = torch.cuda.Stream()
    args = [wide.cuda(), c.pool.cuda(), c.table.cuda(), c.seqlens.cuda()]
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = None
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.out = lib.latent_attention(args[0][..., 32:544], args[0][..., 544:608], args[1], kv, args[2],
                                     args[3], c.scale, out=out.transpose(0, 1)[..., :512], workspace=ws,
                                     dev_status=c.status)
    s.synchronize()
    c.check()
    assert (out[..., 512:] == 3).all()


@pytest.mark.parametrize("kv", KVS)
def test_repeatable_and_back_to_back(kv):
    """Calls back to back on one workspace give the same bits."""
    c = Case([3000, 10, 700, 0, 64], 64, kv, seed=17)
    ws = torch.empty(lib.dsa_latent_attention_workspace(), device="cuda")
    args = (c.q[..., :512].contiguous().cuda(), c.q[..., 512:].contiguous().cuda(), c.pool.cuda(), kv,
            c.table.cuda(), c.seqlens.cuda(), c.scale)
    outs = [lib.latent_attention(*args, workspace=ws) for _ in range(20)]
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


@pytest.mark.parametrize("kv", KVS)
def test_graph_replay_with_other_lengths(kv):
    c = Case([500, 900, 64, 130], 16, kv, seed=18, W=15)
    q, pool, table, lens = c.q.cuda(), c.pool.cuda(), c.table.cuda(), c.seqlens.cuda()
    c.status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.lse = torch.empty((4, 16), device="cuda")
    c.out = torch.empty((4, 16, 512), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(lib.dsa_latent_attention_workspace(), device="cuda")

    def call():
        lib.latent_attention(q[..., :512], q[..., 512:], pool, kv, table, lens, c.scale, out=c.out,
                             lse=c.lse, workspace=ws, dev_status=c.status)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ([500, 900, 64, 130], [0, 901 - 1, 1, 128], [499, 0, 0, 0]):
        c.seqlens = torch.tensor(new, dtype=torch.int32)
        lens.copy_(c.seqlens)
        graph.replay()
        torch.cuda.synchronize()
        c.check()


@pytest.mark.parametrize("kv", KVS)
def test_many_short_rows_again_and_again(kv):
    """Rows of one tile, several per slice: queries and tile change places at every step."""
    c = Case([40] * 300 + [128] * 40, 64, kv, seed=19)
    first = c.run().out.clone()
    c.check(rows=range(0, 340, 11))
    for _ in range(8):
        assert torch.equal(c.run().out, first)
