"""The selection of pages: exact scores, so that the lists are those of the definition, entry by entry."""
import math

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, heads, kv_heads, dim, dtype, seed=0, shared=False, alike=False):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.kv_heads, self.dim, self.R = lens, heads, kv_heads, dim, len(lens)
        rows = [max(lens)] if shared else lens
        used = [ref.pages_of(max(n, 0)) for n in rows]
        pages = sum(used) + 1
        self.W = max(1, max(used))
        perm, at = torch.randperm(pages, generator=g).to(torch.int32), 0
        self.table = torch.full((len(rows), self.W), -1, dtype=torch.int32)
        for r, m in enumerate(used):
            self.table[r, :m] = perm[at:at + m]
            at += m
        shape = (pages, kv_heads, 2, dim)
        if alike:                                           # few kinds of pages: many equal scores
            kinds = torch.randint(-127, 128, (3, kv_heads, 2, dim), generator=g)
            self.bounds = kinds[torch.randint(0, 3, (pages,), generator=g)].to(torch.int8)
            self.unit = torch.full((pages, kv_heads), 0.25)
        else:
            self.bounds = torch.randint(-127, 128, shape, generator=g).to(torch.int8)
            self.unit = torch.exp2(torch.randint(-3, 3, (pages, kv_heads), generator=g).float())
        self.q = torch.randn((self.R, heads, dim), generator=g).to(ref.TYPES[dtype])
        self.seqlens = torch.tensor(lens, dtype=torch.int32)

    def run(self, k, first=1, last=1, q=None):
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.k, self.first, self.last = k, first, last
        out = torch.full((self.R, self.kv_heads, k), 12345, dtype=torch.int32, device="cuda")
        back = lib.block_select(self.q.cuda() if q is None else q, self.bounds.cuda(), self.unit.cuda(), self.table.cuda(),
                                self.seqlens.cuda(), k, first=first, last=last, out=out, dev_status=self.status)
        assert back is out
        self.out = out.cpu()
        return self

    def want(self, r, h):
        n = ref.pages_of(max(self.lens[r], 0))
        page = self.table[0 if self.table.shape[0] == 1 else r, :n].long()
        group = self.heads // self.kv_heads
        found = ref.select(self.q[r, h * group:(h + 1) * group], self.bounds[page, h], self.unit[page, h], self.k,
                           self.first, self.last)
        return found + [-1] * (self.k - len(found))

    def check(self, status=0, rows=None):
        assert int(self.status) == status
        for r in range(self.R) if rows is None else rows:
            for h in range(self.kv_heads):
                assert self.out[r, h].tolist() == self.want(r, h), (r, h)
        return self


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 2), (35, 5), (64, 1), (128, 1)])
@pytest.mark.parametrize("k", [2, 7, 32])
def test_select(dtype, dim, heads, kv_heads, k):
    Case([1, 0, 64, 65, 64 * k, 64 * k + 1, 5000, 20000], heads, kv_heads, dim, dtype, seed=k).run(k).check()


@pytest.mark.parametrize("first,last", [(0, 0), (0, 3), (4, 0), (5, 3), (8, 0), (0, 8)])
@pytest.mark.parametrize("alike", [False, True])
def test_pages_that_are_always_taken(first, last, alike):
    Case([700, 2000, 513, 9000], 8, 2, 64, "bf16", seed=first, alike=alike).run(8, first, last).check()


@pytest.mark.parametrize("k", [1, 3, 64, 100, 333])
def test_equal_scores_from_the_front(k):
    Case([30000, 6400, 6401], 4, 2, 128, "bf16", seed=k, alike=True).run(k, 0, min(k, 1)).check()


def test_all_scores_equal():
    c = Case([4000], 4, 1, 64, "bf16", seed=1)
    c.q[:] = 0
    c.run(9, 0, 0).check()
    assert c.out[0, 0].tolist() == list(range(9))


@pytest.mark.parametrize("k", [16, 600])
def test_long_row(k):
    """The most pages that a row may have, and one list of many."""
    Case([32768 * 64, 100000], 2, 1, 64, "bf16", seed=k).run(k).check()


def test_shared_table():
    Case(list(range(3000, 3100)), 8, 2, 128, "fp16", seed=2, shared=True).run(6).check(rows=range(0, 100, 7))


def test_strided_queries():
    c = Case([3000, 900], 6, 3, 64, "bf16", seed=3)
    wide = torch.full((2, 14, 64), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:14:2] = c.q.cuda()
    c.run(5, q=wide[:, 2:14:2]).check()


def test_special_queries():
    """NaN, infinities, the smallest and the largest numbers."""
    c = Case([3000] * 6, 4, 2, 64, "bf16", seed=4)
    c.q[0, 0, 3] = math.nan
    c.q[1, 1, 5] = math.inf
    c.q[2, 2, 6] = -math.inf
    c.q[3] *= 2.0 ** -133                                  # subnormal
    c.q[4] *= 2.0 ** 120
    c.q[5, :2] = 0
    c.run(7).check()


def test_scores_past_the_largest_float():
    c = Case([3000], 4, 2, 64, "bf16", seed=5)
    c.unit[:] = 2.0 ** 122
    c.run(7).check()


def test_data_errors():
    """A length past the table, pages outside the pool among the row's: no list, a status; others as they are."""
    c = Case([3000, 640, 2000, 300], 4, 2, 64, "bf16", seed=6)
    c.table[1, 3] = 10 ** 7
    c.table[3, 2] = -1                                     # of a row that has all its pages listed
    c.seqlens[0] = c.W * 64 + 1
    c.run(5).check(status=7, rows=[2])
    assert (c.out[[0, 1]] == -1).all()
    c.run(8)
    assert (c.out[[0, 1, 3]] == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 7, 7), (128, 16, 2), (128, 12, 1)])
@pytest.mark.parametrize("low,rows,k", [(1, 400, 3), (1000, 333, 8), (100000, 310, 33), (131000, 306, 700)])
def test_rows_of_a_prompt(dtype, dim, heads, kv_heads, low, rows, k):
    """Many rows that share a table: pages from none to all that the shared kernel has room for."""
    lens = list(range(low - 1, low - 1 + rows))
    lens[rows // 2] = 0
    c = Case(lens, heads, kv_heads, dim, dtype, seed=k, shared=True, alike=k == 8)
    c.run(k).check(rows=sorted({0, 1, rows // 2, rows - 1, *range(0, rows, 37)}))


def test_rows_of_a_prompt_data_errors():
    """A page outside the pool touches the rows that reach it, a length past the table its own."""
    c = Case(list(range(300, 500)), 4, 2, 64, "bf16", seed=7, shared=True)
    c.table[0, 5] = 10 ** 7                                # position 320
    c.seqlens[3] = c.W * 64 + 1
    c.run(4)
    assert int(c.status) == 7
    assert (c.out[3] == -1).all() and (c.out[21:] == -1).all()
    c.check(status=7, rows=[0, 1, 2, 4, 20])


@pytest.mark.parametrize("k", [1, 40, 1024, 1025, 3000])
@pytest.mark.parametrize("alike", [False, True])
def test_lists_of_any_length(k, alike):
    """Rows of one block beside rows of several, lists longer than a block's run and than the joint choice takes."""
    Case([200000, 64 * 256, 64 * 257, 40000, 100, 0], 2, 1, 64, "bf16", seed=k, alike=alike).run(k, 0, 1).check()


def test_bad_page_of_another_block():
    c = Case([100000, 90000], 2, 1, 64, "bf16", seed=8)
    c.table[0, 1400] = -1
    c.run(9).check(status=6, rows=[1])
    assert (c.out[0] == -1).all()


@pytest.mark.parametrize("rows,kv_heads,most", [(70, 2, 1300), (40, 1, 700), (18, 1, 900), (16, 1, 2100), (3, 2, 1100)])
@pytest.mark.parametrize("alike", [False, True])
def test_rows_of_clusters(rows, kv_heads, most, alike):
    """Two, four and eight blocks a row, some of them without a page."""
    lens = [1 + (most * 64 - 1) * (rows - r) // rows * (r % 7 != 3) for r in range(rows)]
    c = Case(lens, 4 * kv_heads, kv_heads, 64, "bf16", seed=rows, alike=alike)
    c.run(20, 2, 3).check(rows=range(0, rows, max(1, rows // 7)))


@pytest.mark.parametrize("dtype,dim,group,kv_heads,rows,most,k", [
    ("bf16", 128, 4, 8, 1030, 22528, 16), ("fp16", 64, 12, 8, 1101, 9001, 5), ("bf16", 128, 1, 2, 4225, 32768, 100),
    ("fp16", 128, 9, 16, 489, 640, 3)])
@pytest.mark.parametrize("alike", [False, True])
def test_many_rows_of_a_shared_table(dtype, dim, group, kv_heads, rows, most, k, alike):
    """32 rows a block, the last block's partly there; rows of no length and of one token between long ones."""
    lens = [0 if r % 11 == 3 else 1 if r % 17 == 5 else max(1, most - rows + 1 + r) for r in range(rows)]
    c = Case(lens, group * kv_heads, kv_heads, dim, dtype, seed=k, shared=True, alike=alike)
    c.run(k).check(rows=sorted({*range(0, rows, rows // 9), 3, 5, 31, 32, rows - 2, rows - 1}))
