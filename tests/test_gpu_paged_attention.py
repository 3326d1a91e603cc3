"""Attention over the paged cache of keys and values against the 64-bit formula, element by element
within the bound that its roundings allow.  Every place without a token holds NaN."""
import itertools
import math

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

PAGE = ref.PAGE
WIDE = 300                                               # a table of so many pages is not a cluster's
KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16")]   # cache, queries


class Case:
    def __init__(self, lens, heads, kv_heads, dim, kv, dtype, layout="head", seed=0, spread=1.0, shared=False,
                 W=None, blocks=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.kv_heads, self.dim, self.kv = lens, heads, kv_heads, dim, kv
        self.dtype, self.R, self.scale, self.blocks = ref.TYPES[dtype], len(lens), dim ** -0.5, blocks
        rows = [max(lens)] if shared else lens
        used = [ref.pages_of(max(n, 0)) for n in rows]
        self.W = W or max(1, max(used))
        pages = sum(used) + 2
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        # entries behind a row's pages hold ids that are not in the pool
        self.table = torch.full((len(rows), self.W), -7, dtype=torch.int32)
        self.pools = ref.Pools(pages, kv_heads, dim, kv, layout)
        at = 0
        for r, n in enumerate(rows):
            n, m = max(n, 0), used[r]
            self.table[r, :m] = perm[at:at + m]
            at += m
            t = torch.arange(n)
            page, slot = self.table[r].long()[t // PAGE], t % PAGE
            k, v = (torch.randn((n, kv_heads, dim), generator=g) *
                    torch.exp(spread * torch.randn((n, kv_heads, 1), generator=g)) for _ in range(2))
            if n:
                self.pools.put(page, slot, k.to(self.dtype), v.to(self.dtype))
        self.q = torch.randn((self.R, heads, dim), generator=g).to(self.dtype)
        self.seqlens = torch.tensor(lens, dtype=torch.int32)

    def run(self, q=None, out=None, **more):
        k, v, ks, vs = self.pools.cuda()
        blocks = None if self.blocks is None else self.blocks.cuda()
        if blocks is not None and self.blocks.stride(1) == 0:
            blocks = self.blocks[:, :1].cuda().expand(self.blocks.shape)
        q = self.q.cuda() if q is None else q
        self.out = torch.full(self.q.shape, 3.0, dtype=self.dtype, device="cuda") if out is None else out
        self.lse = torch.full((self.R, self.heads), 3.0, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        floats = lib.dsa_paged_attention_workspace(self.heads, self.kv_heads, self.dim)
        back = lib.paged_attention(q, k, v, self.table.cuda(), self.seqlens.cuda(), self.scale, blocks=blocks,
                                   k_scale=ks, v_scale=vs, out=self.out, lse=self.lse,
                                   workspace=torch.full((floats,), math.nan, device="cuda"),
                                   dev_status=self.status, **more)
        assert back is self.out
        return self

    def tokens(self, r, head):
        n, row = self.lens[r], self.table[0 if self.table.shape[0] == 1 else r].long()
        t = torch.arange(max(n, 0))
        if self.blocks is not None:
            t = [torch.arange(b * PAGE, min((b + 1) * PAGE, n)) for b in self.blocks[r, head].tolist()
                 if 0 <= b < ref.pages_of(n)]
            t = torch.cat(t) if t else torch.arange(0)
        return row[t // PAGE], t % PAGE

    def check(self, status=0, rows=None):
        torch.cuda.synchronize()
        assert int(self.status) == status
        out, lse = self.out.double().cpu(), self.lse.double().cpu()
        group = self.heads // self.kv_heads
        for r in range(self.R) if rows is None else rows:
            for h in range(self.kv_heads):
                page, slot = self.tokens(r, h)
                k, v = self.pools.get(page, slot)
                hs = slice(h * group, (h + 1) * group)
                want, want_lse, bound, lse_bound = ref.attention_row(
                    self.q[r, hs].double(), k[:, h:h + 1], v[:, h:h + 1], self.scale, self.kv, self.dtype)
                off = (out[r, hs] - want).abs()
                assert (off <= bound).all(), (r, h, float((off / bound.clamp(min=1e-300)).max()))
                assert torch.equal(lse[r, hs].isneginf(), want_lse.isneginf())
                far = torch.where(want_lse.isneginf(), 0.0, (lse[r, hs] - want_lse).abs())
                assert (far <= lse_bound).all(), (r, h, float(far.max()))
        return self


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(8, 1), (35, 5)])
@pytest.mark.parametrize("W", [None, WIDE])
def test_one_page_and_less(kv, dtype, dim, heads, kv_heads, W):
    Case([1, 2, 15, 16, 17, 33, 63, 64, 0], heads, kv_heads, dim, kv, dtype, seed=1, W=W).run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("layout", ["head", "token", "both", "wide"])
@pytest.mark.parametrize("W", [None, WIDE])
def test_layouts(kv, dtype, dim, layout, W):
    Case([65, 0, 200, 129, 640], 12, 3, dim, kv, dtype, layout, seed=2, W=W).run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 7, 8, 9, 16, 17, 24, 32, 33, 40, 64, 100])
@pytest.mark.parametrize("W", [None, WIDE])
def test_groups(kv, dtype, dim, group, W):
    """Query heads of a key head: less than a tile, whole ones, more than a CTA takes."""
    Case([100, 700], 2 * group, 2, dim, kv, dtype, "token", seed=group, W=W).run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("rows,lens", [(1, [500]), (1, [512]), (1, [2]), (2, [4000, 130]), (9, [64, 0, 640, 1, 1024]), (20, [500, 0, 9]),
                                       (38, [70, 256])])
def test_rows_of_a_cluster(kv, dtype, rows, lens):
    """Clusters of all sizes, with CTAs that have no page, and rows of one CTA or none."""
    lens = (lens * rows)[:rows]
    Case(lens, 20, 4, 128, kv, dtype, seed=rows).run().check()
    Case(lens, 8, 4, 64, kv, dtype, seed=rows).run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 16, 2), (64, 40, 1)])
def test_long_rows(kv, dtype, dim, heads, kv_heads):
    """Rows that many CTAs share, beside short ones and empty ones."""
    Case([20000, 3, 0, 5000, 64, 0, 9001], heads, kv_heads, dim, kv, dtype, seed=3).run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("rows,heads", [(1, 4), (37, 4), (152, 2), (305, 8), (700, 2)])
def test_many_rows(kv, dtype, rows, heads):
    g = torch.Generator().manual_seed(rows)
    lens = torch.randint(0, 300, (rows,), generator=g).tolist()
    lens[-1] = 0 if rows > 1 else 5
    Case(lens, heads, 2, 64, kv, dtype, seed=rows).run().check(rows=range(0, rows, max(1, rows // 60)))


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("k", [1, 5, 32, 33, 70, 128, 129, 200])
def test_lists(kv, dtype, k):
    """Lists in any order, with holes, entries past the row, a page twice, none at all; a list a head."""
    lens, H = [1000, 64, 0, 4000, 1, 2300], 3
    g = torch.Generator().manual_seed(k)
    blocks = torch.full((len(lens), H, k), -1, dtype=torch.int32)
    for r, h in itertools.product(range(len(lens)), range(H)):
        n = ref.pages_of(lens[r])
        some = torch.randperm(max(n, 1), generator=g)[:k].to(torch.int32)
        blocks[r, h, :some.numel()] = some
    blocks = blocks[..., torch.randperm(k, generator=g)]
    blocks[0, 0] = -1
    blocks[0, 1, 0] = 16                                   # the first past the row
    blocks[0, 2, -1] = 2 ** 31 - 1
    if k > 4:
        blocks[3, 0, :4] = 7
        blocks[3, 1, 1:] = -5
    Case(lens, 12, H, 128, kv, dtype, seed=k, blocks=blocks).run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
def test_one_list_for_all_heads(kv, dtype):
    blocks = torch.tensor([[0, 3, 9, 11], [1, 2, 4, -1]], dtype=torch.int32)[:, None].expand(2, 4, 4)
    c = Case([750, 300], 8, 4, 64, kv, dtype, "token", seed=4, blocks=blocks)
    assert c.blocks.stride(1) == 0
    c.run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("listed", [False, True])
def test_shared_table(kv, dtype, listed):
    """A prompt's tokens: one table row, causal lengths, every token its own pages."""
    lens = list(range(960, 1060))
    blocks = None
    if listed:
        g = torch.Generator().manual_seed(5)
        blocks = torch.stack([torch.stack([torch.randperm(15, generator=g)[:5].sort().values for _ in range(2)])
                              for _ in lens]).to(torch.int32)
    Case(lens, 8, 2, 128, kv, dtype, seed=5, shared=True, blocks=blocks).run().check(rows=range(0, 100, 9))


@pytest.mark.parametrize("kv,dtype", KINDS)
def test_strided_queries_and_results(kv, dtype):
    c = Case([300, 77, 0], 6, 3, 128, kv, dtype, seed=6)
    wide = torch.full((3, 14, 128), math.nan, dtype=c.dtype, device="cuda")
    wide[:, 2:14:2] = c.q.cuda()
    out = torch.full((6, 7, 136), 5.0, dtype=c.dtype, device="cuda")
    view = out[::2, :6, :128]
    c.run(q=wide[:, 2:14:2], out=view).check()
    assert (out[1::2] == 5).all() and (out[:, 6] == 5).all() and (out[..., 128:] == 5).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("power", [-40, -120])
@pytest.mark.parametrize("W", [None, WIDE])
def test_fp8_scales_apart(dtype, power, W):
    """Value scales from 2^power to 1 within a row: tokens of large values beside small and zero ones."""
    c = Case([500], 8, 1, 128, "fp8", dtype, seed=7, spread=0.0, W=W)
    page, slot = c.tokens(0, 0)
    t = torch.arange(500)
    c.pools.v_scale[page, 0, slot] = torch.where(t % 3 == 0, 2.0 ** power, 1.0)
    zero = t % 7 == 1                                        # zeros with the smallest scale, as the store gives them
    c.pools.v.view(torch.uint8)[page[zero], slot[zero]] = 0
    c.pools.v_scale[page[zero], 0, slot[zero]] = 2.0 ** -126
    c.run().check()
    # small tokens alone keep their precision
    c.pools.v_scale[page, 0, slot] = 2.0 ** power
    c.run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("factor", [2.0 ** -60, 30.0, 2000.0])
@pytest.mark.parametrize("W", [None, WIDE])
def test_scores_of_any_size(kv, dtype, factor, W):
    """From a uniform softmax to one token that takes all."""
    if dtype == "fp16" and factor < 1:
        factor = 2.0 ** -14
    c = Case([777, 64], 8, 2, 64, kv, dtype, seed=8, spread=0.0, W=W)
    c.q = (c.q.double() * factor).to(c.dtype)
    c.run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
def test_queries_of_nan(kv, dtype):
    c = Case([130, 130, 130], 4, 2, 64, kv, dtype, seed=9)
    c.q[1, 2] = math.nan                                     # one head of one row
    c.run()
    torch.cuda.synchronize()
    assert c.out[1, 2].isnan().all() and c.lse[1, 2].isnan()
    assert c.out[1, [0, 1, 3]].isfinite().all() and c.out[[0, 2]].isfinite().all()
    c.check(rows=[0, 2])


@pytest.mark.parametrize("kv,dtype", KINDS)
def test_nan_of_a_visible_token(kv, dtype):
    c = Case([130, 70], 4, 2, 128, kv, dtype, seed=10)
    page, slot = c.tokens(0, 0)
    ref.bytes_of(c.pools.v)[page[129], slot[129], 1, 5] = 0x7f if kv == "fp8" else math.nan
    c.run()
    torch.cuda.synchronize()
    bad = c.out.isnan().cpu()
    assert bad[0, 2:, 5].all() and int(bad.sum()) == 2
    c.check(rows=[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("values", [False, True])
def test_nan_scales_of_a_visible_token(dtype, values):
    c = Case([130, 70], 4, 2, 128, "fp8", dtype, seed=17)
    page, slot = c.tokens(0, 0)
    (c.pools.v_scale if values else c.pools.k_scale)[page[100], 1, slot[100]] = math.nan
    c.run()
    torch.cuda.synchronize()
    assert c.out[0, 2:].isnan().all() and c.out[0, :2].isfinite().all()
    c.check(rows=[1])


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("W", [None, WIDE])
def test_data_errors(kv, dtype, W):
    """A length past the table, pages outside the pool: NaN, a status, and the other rows as they are."""
    c = Case([300, 200, 64, 1000], 8, 2, 128, kv, dtype, seed=11, W=W)
    c.table[1, 2] = 10 ** 6
    c.seqlens[2] = c.W * PAGE + 1
    c.run()
    torch.cuda.synchronize()
    assert int(c.status) == 7
    assert c.out[1:3].isnan().all() and c.lse[1:3].isnan().all()
    c.check(status=7, rows=[0, 3])
    c.seqlens[2] = 64
    c.table[1, 2] = -1
    c.run().check(status=6, rows=[0, 2, 3])
    assert c.out[1].isnan().all()


def test_bad_page_of_a_row_that_ctas_share():
    c = Case([9000, 100], 8, 2, 128, "bf16", "bf16", seed=12)
    c.table[0, 77] = -3
    c.run().check(status=6, rows=[1])
    assert c.out[0].isnan().all() and c.lse[0].isnan().all()


def test_bad_page_that_no_list_names():
    blocks = torch.tensor([0, 2], dtype=torch.int32).expand(1, 2, 2)
    c = Case([190], 8, 2, 128, "bf16", "bf16", seed=13, blocks=blocks)
    c.table[0, 1] = -3
    c.run().check()


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("lens", [[5000, 64, 700, 12000], [900, 64, 3, 1000]])
def test_same_bits_every_time(kv, dtype, lens):
    c = Case(lens, 16, 2, 128, kv, dtype, seed=14)
    first = c.run().out.clone(), c.lse.clone()
    for _ in range(5):
        c.run()
        assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("lens,heads,W", [([1000], 8, None), ([1000, 0, 70], 70, None), ([30000], 40, None), ([70, 9000, 0, 300] * 9, 24, WIDE)])
def test_results_in_the_queries_place(kv, dtype, lens, heads, W):
    c = Case(lens, heads, 2, 64, kv, dtype, seed=len(lens), W=W)
    q = c.q.cuda()
    c.run(q=q, out=q).check()


def test_no_rows_and_allocated_outputs():
    c = Case([100], 4, 2, 64, "bf16", "bf16", seed=15)
    k, v, _, _ = c.pools.cuda()
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    out = lib.paged_attention(c.q.cuda()[:0], k, v, c.table.cuda(), none, c.scale)
    assert out.shape == (0, 4, 64)
    c.run()
    out = lib.paged_attention(c.q.cuda(), k, v, c.table.cuda(), c.seqlens.cuda(), c.scale)
    assert torch.equal(out, c.out)


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31 from the pool's start."""
    free, _ = torch.cuda.mem_get_info()
    pages, H, D = 2 ** 31 // (2 * 64 * 128) + 40, 2, 128
    if free < 3 * pages * H * 64 * D * 2:
        pytest.skip("not enough memory")
    c = Case([200], 4, H, D, "bf16", "bf16", seed=16)
    k, v, _, _ = c.pools.cuda()
    pool = torch.empty((pages, H, PAGE, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    far = torch.arange(pages - k.shape[0], pages, device="cuda")
    pool[far] = k
    values = torch.empty((pages, H, PAGE, D), dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    values[far] = v
    c.run()
    out = lib.paged_attention(c.q.cuda(), pool, values, (c.table + (pages - k.shape[0])).cuda(), c.seqlens.cuda(), c.scale)
    assert torch.equal(out, c.out)
    c.check()
