"""Edges of the calls on the paged cache of keys and values."""
import math

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import paged_ref as ref
from tests.test_gpu_block_select import Case as Selection
from tests.test_gpu_paged_attention import KINDS, WIDE, Case

pytestmark = pytest.mark.gpu

PAGE = ref.PAGE


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- a free list that ends ---------------------------------------------------------------

def slots_by_contract(lengths, new, free, table, n):
    """Requests in order; one that wants more pages than are left takes none and leaves them to the next."""
    table, slots, positions, seqlens, cu, at, status = [list(r) for r in table], [], [], [], [0], 0, 0
    for b, (c, m) in enumerate(zip(lengths, new)):
        have, want = ref.pages_of(c), ref.pages_of(c + m)
        good = want == have or want - have <= len(free) - at
        if not good:
            status = 6
        else:
            table[b][have:want] = free[at:at + want - have]
            at += want - have
        for p in range(c, c + m):
            slots.append(table[b][p // PAGE] * PAGE + p % PAGE if good else -1)
            positions.append(p if good else 0)
        seqlens.append(c + m if good else 0)
        cu.append(cu[-1] + m)
    rest = n - len(slots)
    return table, slots + [-1] * rest, positions + [0] * rest, seqlens, cu, at, status


def check_slots(lengths, new, free):
    W, n, at, table = max(1, *(ref.pages_of(c + m) for c, m in zip(lengths, new))), sum(new) + 3, 5000, []
    for c in lengths:
        held = ref.pages_of(c)
        table.append(list(range(at, at + held)) + [-1] * (W - held))
        at += held
    there, status = int32(table), int32([0])
    slots, positions, seqlens, cu, used = lib.request_slots(int32(lengths), int32(new), int32(free), there, n, dev_status=status)
    got = there.tolist(), slots.tolist(), positions.tolist(), seqlens.tolist(), cu.tolist(), int(used), int(status)
    assert got == slots_by_contract(lengths, new, free, table, n)


@pytest.mark.parametrize("lengths,new,pages", [
    ([0, 0], [12 * 64, 1], 10), ([0, 60, 64], [700, 10, 1], 10), ([0, 5, 0, 0, 64], [65, 3, 64, 65, 1], 2),
    ([64, 0, 0, 0, 0], [1, 129, 128, 129, 64], 4), ([0, 0, 0], [64, 65, 64], 0), ([0, 0, 0], [128, 64, 64], 1)])
def test_slots_behind_a_refused_request(lengths, new, pages):
    check_slots(lengths, new, [70 + 3 * i for i in range(pages)])


@pytest.mark.parametrize("requests,pages,high", [(64, 40, 200), (1024, 900, 150), (1030, 700, 300), (2500, 2400, 200), (3000, 1, 90)])
def test_slots_behind_many_refused_requests(requests, pages, high):
    """Free lists that end in the first, a later or no chunk of requests, those that fit between those that do not."""
    g = torch.Generator().manual_seed(requests)
    lengths = torch.randint(0, 130, (requests,), generator=g).tolist()
    new = torch.randint(0, high, (requests,), generator=g).tolist()
    check_slots(lengths, new, torch.randperm(4000, generator=g)[:pages].tolist())


# ---- keys far apart ------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "fp16", "fp8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_boxes_of_channels_far_apart(kv, dim):
    """A channel so much smaller than the page's largest that its quotient underflows still lies in the box."""
    x = torch.randn((4, PAGE, 1, dim), generator=torch.Generator().manual_seed(dim))
    x[:, :, 0, 1], x[:, :, 0, 2] = x[:, :, 0, 1].abs() + 1, -x[:, :, 0, 2].abs() - 1
    small = 2.0 ** -60 if kv == "bf16" else 2.0 ** -20
    x = (x * small).to(ref.TYPES["bf16" if kv == "fp8" else kv])
    large = float(torch.finfo(x.dtype).max)
    for page in range(1, 4):                                   # of one token, as it is stored
        x[page, 7] = 0
        x[page, 7, 0, 5] = (0, large, -large, math.inf if kv != "fp8" else large / 3)[page]
    pools = ref.Pools(4, 1, dim, kv)
    page, slot = torch.arange(4 * PAGE) // PAGE, torch.arange(4 * PAGE) % PAGE
    pools.put(page, slot, x.flatten(0, 1), x.flatten(0, 1))
    if kv == "fp8":
        pools.k_scale[1:, 0, torch.arange(PAGE) != 7] *= 2.0 ** -60
    k, _, ks, _ = pools.cuda()
    bounds = torch.zeros((4, 1, 2, dim), dtype=torch.int8, device="cuda")
    unit = torch.zeros((4, 1), device="cuda")
    lib.block_bounds(k, torch.arange(4, dtype=torch.int32, device="cuda")[None], None, int32([4 * PAGE]), 4 * PAGE, bounds, unit,
                     k_scale=ks)
    for p in range(4):
        keys, _ = pools.get(torch.full((PAGE,), p), torch.arange(PAGE))
        want, scale = ref.box(keys[:, 0])
        assert float(unit[p, 0]) == scale
        assert torch.equal(bounds[p, 0].cpu(), want), p


# ---- queries and scales at the ends of their range ------------------------------------------

@pytest.mark.parametrize("power", [-110, -60, 60, 100, 120])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("W", [None, WIDE])
def test_fp8_queries_against_their_keys(power, dim, W):
    """Queries of 2^power with keys of 2^-power: scores of ordinary size."""
    c = Case([300, 64], 20, 2, dim, "fp8", "bf16", seed=power + 200, spread=0.5, W=W)
    c.q = (c.q.double() * 2.0 ** power).to(c.dtype)
    c.pools.k_scale *= 2.0 ** -power
    c.run().check()


@pytest.mark.parametrize("W", [None, WIDE])
def test_fp8_smallest_queries(W):
    """bf16's subnormal numbers keep their bits beside the largest keys."""
    c = Case([200], 8, 2, 64, "fp8", "bf16", seed=1, spread=0.0, W=W)
    c.q = (c.q.double() * 2.0 ** -128).to(c.dtype)
    c.pools.k_scale *= 2.0 ** 124
    c.run().check()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,pages,every", [(1, 24, 3), (608, 2, 2)])
def test_fp8_largest_value_scales(dtype, rows, pages, every):
    """Small codes under scales near 2^127, on tokens whose scores are a little above those before them,
    wherever a row's pages are shared out."""
    n = pages * PAGE
    c = Case([n] * rows, 8, 1, 64, "fp8", dtype, seed=2, spread=0.0)
    c.scale = 1.0
    c.q[:] = 0
    c.q[..., 0] = 8.0
    late = torch.arange(n) // PAGE % every == every - 1
    key = torch.zeros((n, 1, 64))
    key[late, 0, 0] = 0.6                                       # 7 in log2 units: no reason for a new reference
    g = torch.Generator().manual_seed(3)
    top = 126 if dtype == "bf16" else 14                        # results that the type has
    for r in range(rows):
        page, slot = c.tokens(r, 0)
        value = (torch.rand((n, 1, 64), generator=g) + 0.25).to(torch.float8_e4m3fn)
        c.pools.put(page, slot, key, key)
        c.pools.v.view(torch.uint8)[page, slot] = value.view(torch.uint8)
        c.pools.v_scale[page, 0, slot] = torch.where(late, 2.0 ** top, 1.0)
    c.run().check(rows=range(0, rows, 101))


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 26, 2.0 ** 33])
@pytest.mark.parametrize("lens,W", [([900], None), ([900, 64, 9000], WIDE)])
def test_one_token_takes_all(kv, dtype, size, lens, W):
    """Scores far past the steps of 1 that an fp32 has: the token with the largest is the result, whatever
    the value scales beside it.  Off by two roundings of 16 bits (the result's, the weight's) and, of
    2^-18 each at most, a few steps of exponents up to 2^7."""
    c = Case(lens, 8, 2, 64, kv, dtype, seed=30, spread=0.0, W=W)
    c.scale = size * (1 + 2.0 ** -9 / 3)                        # no power of two
    c.q[:] = 0
    c.q[..., 5] = 1.0 + 2.0 ** -7
    g = torch.Generator().manual_seed(31)
    for r, n in enumerate(lens):
        page, slot = c.tokens(r, 0)
        best = torch.randint(0, n, (1,), generator=g)
        key = torch.zeros((n, 2, 64))
        key[:, :, 5] = 0.5 + 0.25 * torch.rand((n, 1), generator=g)
        key[best, :, 5] = 1.375
        value = torch.randn((n, 2, 64), generator=g) * torch.exp2(torch.randint(-6, 7, (n, 2, 1), generator=g).float())
        c.pools.put(page, slot, key.to(c.dtype), value.to(c.dtype))
        c.best = [*getattr(c, "best", []), (page[best], slot[best])]
    c.run()
    torch.cuda.synchronize()
    assert int(c.status) == 0
    step = torch.finfo(c.dtype).eps / 2 + (2.0 ** -8 if kv == "bf16" else 2.0 ** -11) + 2.0 ** -14
    for r, at in enumerate(c.best):
        _, value = c.pools.get(*at)
        want = value[0].repeat_interleave(4, 0)
        off = (c.out[r].double().cpu() - want).abs()
        assert (off <= step * want.abs() + 2.0 ** -25).all(), (r, float((off / want.abs()).max()))


# ---- the widest shared table -----------------------------------------------------------------

@pytest.mark.parametrize("dtype,dim,heads,kv_heads", [("bf16", 64, 4, 2), ("fp16", 128, 8, 1)])
@pytest.mark.parametrize("k", [5, 700])
def test_widest_table_that_rows_share(dtype, dim, heads, kv_heads, k):
    """Exactly the 2,048 pages that a block of 16 rows has room for, the last row's keys before the page ids."""
    rows = 330
    lens = list(range(131072 - rows + 1, 131072 + 1))
    c = Selection(lens, heads, kv_heads, dim, dtype, seed=k, shared=True)
    assert c.W == 2048
    c.run(k).check(rows=[0, 1, 14, 15, 16, 200, rows - 2, rows - 1])


# ---- what the header says of lists and scores without a finite number ---------------------------

@pytest.mark.parametrize("kv", ["bf16", "fp16"])
@pytest.mark.parametrize("W", [None, WIDE])
def test_scores_all_minus_infinity(kv, W):
    c = Case([130, 300], 8, 2, 64, kv, kv, seed=20, W=W)
    page, slot = c.tokens(0, 0)
    c.pools.k[page, slot, 1, 3] = -math.inf
    c.q[..., 3] = 1.0
    c.run().check(rows=[1])
    assert (c.out[0, 4:] == 0).all() and c.lse[0, 4:].isneginf().all()
    assert c.out[0, :4].isfinite().all() and c.lse[0, :4].isfinite().all()


def test_list_of_a_bad_table():
    """A table with a page outside the pool: -1 from the selection, zeros from the attention, and the status."""
    c = Case([700, 500], 4, 2, 64, "bf16", "bf16", seed=21)
    c.table[0, 2] = 10 ** 6
    pages = c.pools.k.shape[0]
    bounds = torch.ones((pages, 2, 2, 64), dtype=torch.int8, device="cuda")
    status = int32([0])
    c.blocks = lib.block_select(c.q.cuda(), bounds, torch.ones((pages, 2), device="cuda"), c.table.cuda(), c.seqlens.cuda(), 4,
                                dev_status=status).cpu()
    assert int(status) == 6 and (c.blocks[0] == -1).all() and (c.blocks[1] >= 0).all()
    c.run().check()
    assert (c.out[0] == 0).all() and c.lse[0].isneginf().all()
