"""The paged cache of keys and values: slots from lengths, the store and the pages' boxes, against
the definitions, value by value."""
import math

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

PAGE = ref.PAGE
KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("fp8", "bf16"), ("fp8", "fp16")]   # cache, tokens


def int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ---- slots ----------------------------------------------------------------------------

def run_slots(lengths, new, free, table, n, wide=0):
    W = len(table[0])
    full = torch.full((len(table), W + wide), -9, dtype=torch.int32, device="cuda")
    full[:, :W] = int32(table)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots, positions, seqlens, cu, used = lib.request_slots(
        int32(lengths), int32(new), int32(free), full[:, :W], n, dev_status=status)
    assert (full[:, W:] == -9).all()
    return full[:, :W].tolist(), slots.tolist(), positions.tolist(), seqlens.tolist(), cu.tolist(), int(used), int(status)


def check_slots(lengths, new, free, table, n, **more):
    assert run_slots(lengths, new, free, table, n, **more) == ref.request_slots(lengths, new, free, table, n)


def tables(lengths, W, at=1000):
    rows = []
    for c in lengths:
        held = ref.pages_of(max(c, 0))
        rows.append(list(range(at, at + held))[:W] + [-1] * (W - min(held, W)))
        at += held
    return rows


@pytest.mark.parametrize("lengths,new", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([63], [2]), ([5], [0]), ([0], [0]), ([0, 0, 0], [64, 65, 63]),
    ([10, 64, 128, 1, 0], [0, 0, 1, 130, 7]), ([191, 192, 193], [1, 1, 1]),
])
@pytest.mark.parametrize("rest", [0, 1, 300])
def test_slots_small(lengths, new, rest):
    check_slots(lengths, new, list(range(50)), tables(lengths, 6), sum(new) + rest, wide=3)


@pytest.mark.parametrize("requests,high", [(64, 1), (23, 700), (1000, 3), (1025, 2), (3000, 5), (1, 20000)])
def test_slots_many(requests, high):
    g = torch.Generator().manual_seed(requests)
    lengths = torch.randint(0, 400, (requests,), generator=g).tolist()
    new = torch.randint(0, high + 1, (requests,), generator=g).tolist()
    free = torch.randperm(20000, generator=g).tolist()
    check_slots(lengths, new, free, tables(lengths, ref.pages_of(400 + high), 30000), sum(new) + 5)


def test_slots_data_errors():
    """Bad lengths, a free list that ends, pages out of range, too few rows."""
    lengths, new = [10, -1, 600, 64, 0, 20], [5, 3, 100, -2, 70, 1]
    table = tables([10, 0, 600, 64, 0, 20], 10)
    check_slots(lengths, new, [1, 2, 3], table, 190)
    check_slots([64, 64, 64, 64], [64, 1, 65, 1], [5, 6], tables([64] * 4, 4), 131)      # the third needs two, has none
    check_slots([64, 0], [1, 2], [], tables([64, 0], 2), 3)
    check_slots([0, 0, 64], [1, 1, 1], [-4, 2 ** 30, 7], tables([0, 0, 64], 2), 3)
    check_slots([3, 60], [5, 10], [9, 8], tables([3, 60], 2), 8)                          # seven rows too few


def test_slots_some_outputs():
    """The nullable outputs, at the C level."""
    lengths, new, free = int32([64, 3]), int32([2, 1]), int32([8, 9])
    table = int32([[4, -1], [5, -1]])
    slots = torch.full((5,), -7, dtype=torch.int32, device="cuda")
    assert lib.dsa_request_slots(lengths, new, 2, free, 2, table, 2, 2, 64, 5, slots, None, None, None, None) == 0
    assert slots.tolist() == [512, 513, 323, -1, -1] and table.tolist() == [[4, 8], [5, -1]]


def test_slots_without_requests():
    none = int32([])
    slots, positions, seqlens, cu, used = lib.request_slots(none, none, none, torch.empty((0, 3), dtype=torch.int32, device="cuda"), 3)
    assert slots.tolist() == [-1] * 3 and positions.tolist() == [0] * 3 and cu.tolist() == [0] and used.tolist() == [0]
    assert seqlens.numel() == 0


# ---- store ----------------------------------------------------------------------------

def same(x, y):
    """Equal bits, NaN like NaN."""
    x, y = (ref.bytes_of(t).cpu() for t in (x, y))
    if x.dtype.is_floating_point:
        return torch.equal(x.isnan(), y.isnan()) and torch.equal(torch.nan_to_num(x), torch.nan_to_num(y))
    return torch.equal(x, y)


@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("layout", ["head", "token", "both", "wide"])
@pytest.mark.parametrize("n,heads", [(1, 1), (70, 3), (333, 8)])
def test_store(kv, dtype, dim, layout, n, heads):
    """Every slot that is named gets its token, whatever the magnitude; all others stay as they are."""
    g = torch.Generator().manual_seed(n)
    pages = ref.pages_of(n) + 2
    pools = ref.Pools(pages, heads, dim, kv, layout)
    k, v, ks, vs = pools.cuda()
    x = torch.randn((n, 2 * heads, dim), generator=g) * torch.exp2(torch.randint(-20, 12, (n, 2 * heads, 1), generator=g).float())
    x = x.to(ref.TYPES[dtype])
    slots = torch.randperm(pages * PAGE, generator=g)[:n].to(torch.int32)
    skip = torch.rand(n, generator=g) < 0.1
    keep = (~skip).nonzero()[:, 0]
    pools.put(slots[keep].long() // PAGE, slots[keep].long() % PAGE, x[keep, :heads], x[keep, heads:])
    slots[skip] = -3
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    there = x.cuda()
    lib.kv_store(there[:, :heads], there[:, heads:], slots.cuda(), k, v, k_scale=ks, v_scale=vs, dev_status=status)
    assert int(status) == 0
    assert same(k, pools.k) and same(v, pools.v)
    if kv == "fp8":
        assert same(ks, pools.k_scale) and same(vs, pools.v_scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_store_of_special_values(dtype):
    t = ref.TYPES[dtype]
    tiny = float(torch.finfo(t).smallest_normal)
    x = torch.zeros((9, 1, 64), dtype=t)
    x[1] = tiny / 4                                            # subnormal
    x[2, 0, 3], x[2, 0, 4] = math.inf, 2.0
    x[3, 0, 5], x[3, 0, 6] = math.nan, -3.0
    x[4] = -math.inf
    x[5] = math.nan
    x[6, 0, :2] = torch.tensor([448.0, -1.0])
    x[7, 0, :2] = torch.tensor([450.0, 0.001])
    x[8] = float(torch.finfo(t).max)
    pools = ref.Pools(1, 1, 64, "fp8")
    k, v, ks, vs = pools.cuda()
    slots = torch.arange(9, dtype=torch.int32)
    lib.kv_store(x.cuda(), -x.cuda(), slots.cuda(), k, v, k_scale=ks, v_scale=vs)
    pools.put(torch.zeros(9, dtype=torch.long), slots.long(), x, -x)
    # a NaN's sign is nobody's
    clear = lambda c: torch.where((c & 0x7f) == 0x7f, 0x7f, c)                  # noqa: E731
    for got, want in ((k, pools.k), (v, pools.v)):
        assert torch.equal(clear(got.view(torch.uint8).cpu()), clear(want.view(torch.uint8)))
    assert same(ks, pools.k_scale) and same(vs, pools.v_scale)


def test_store_past_the_pool():
    pools = ref.Pools(2, 2, 64, "bf16")
    k, v, _, _ = pools.cuda()
    x = torch.ones((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.kv_store(x, x, int32([128, 5, 2 ** 31 - 1]), k, v, dev_status=status)
    assert int(status) == 6
    assert (k[0, 5] == 1).all() and int(k.isfinite().sum()) == 128


# ---- boxes ------------------------------------------------------------------------------

@pytest.mark.parametrize("kv,dtype", KINDS)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("layout", ["head", "wide"])
@pytest.mark.parametrize("hint", [1, 40, 1000])
def test_boxes(kv, dtype, dim, layout, hint):
    """Pages from `starts` on, masked places NaN, others untouched; the hint of the new tokens only shapes the launch."""
    lens, starts, H = [1, 64, 0, 200, 130, 700, 65], [0, 0, 0, 130, 130, 64, -5], 3
    g = torch.Generator().manual_seed(dim)
    pages = sum(ref.pages_of(n) for n in lens) + 1
    pools = ref.Pools(pages, H, dim, kv, layout)
    table = torch.full((len(lens), 12), 10 ** 8, dtype=torch.int32)
    perm, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    for r, n in enumerate(lens):
        m = ref.pages_of(n)
        table[r, :m] = perm[at:at + m]
        at += m
        t = torch.arange(n)
        if n:
            x = torch.randn((n, H, dim), generator=g) * torch.exp2(torch.randint(-12, 8, (1, H, 1), generator=g).float())
            pools.put(table[r].long()[t // PAGE], t % PAGE, x.to(ref.TYPES[dtype]), x.to(ref.TYPES[dtype]))
    bounds = torch.full((pages, H, 2, dim), 77, dtype=torch.int8)
    unit = torch.full((pages, H), -1.0)
    got, got_unit, status = bounds.cuda(), unit.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    k, _, ks, _ = pools.cuda()
    lib.block_bounds(k, table.cuda(), int32(starts), int32(lens), hint, got, got_unit, k_scale=ks, dev_status=status)
    for r, n in enumerate(lens):
        for b in range(max(starts[r], 0) // PAGE, ref.pages_of(n)) if starts[r] < n else ():
            page, t = int(table[r, b]), torch.arange(b * PAGE, min(n, (b + 1) * PAGE))
            keys, _ = pools.get(torch.full_like(t, page), t % PAGE)
            for h in range(H):
                bounds[page, h], unit[page, h] = ref.box(keys[:, h])
    assert int(status) == 0
    assert torch.equal(got.cpu(), bounds) and torch.equal(got_unit.cpu(), unit)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_boxes_of_special_keys(dtype):
    t = ref.TYPES[dtype]
    pools = ref.Pools(6, 1, 64, dtype)
    x = torch.randn((6, PAGE, 1, 64), generator=torch.Generator().manual_seed(3)).to(t)
    x[0, 3, 0, 4] = math.nan                                    # passed over
    x[1, :, 0, 7] = math.nan                                    # no number: 0
    x[2, 1, 0, 8] = math.inf
    x[3] = 0
    x[4] = float(torch.finfo(t).smallest_normal) / 8            # subnormal
    x[5, 9, 0, 1], x[5, 10, 0, 2] = -float(torch.finfo(t).max), -math.inf
    pools.k[:] = x
    k, _, _, _ = pools.cuda()
    bounds = torch.zeros((6, 1, 2, 64), dtype=torch.int8, device="cuda")
    unit = torch.zeros((6, 1), device="cuda")
    lib.block_bounds(k, torch.arange(6, dtype=torch.int32, device="cuda"), None, int32([6 * PAGE]), 6 * PAGE, bounds, unit)
    for p in range(6):
        want, scale = ref.box(x[p, :, 0].double())
        assert torch.equal(bounds[p, 0].cpu(), want), p
        assert float(unit[p, 0]) == scale


def test_boxes_data_errors():
    pools = ref.Pools(3, 2, 64, "bf16")
    pools.k[:] = 1
    k, _, _, _ = pools.cuda()
    bounds = torch.full((3, 2, 2, 64), 9, dtype=torch.int8, device="cuda")
    unit, status = torch.zeros((3, 2), device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    table = int32([[0, -2], [3, 1], [2, 2]])
    lib.block_bounds(k, table, None, int32([128, 128, 129]), 128, bounds, unit, dev_status=status)
    assert int(status) == 7
    assert (bounds[:2] == 64).all() and (bounds[2] == 9).all()


@pytest.mark.parametrize("kv,dim,hint", [("bf16", 64, 3000), ("fp8", 128, 3000), ("fp16", 128, 1), ("fp8", 64, 100)])
def test_boxes_of_many_requests(kv, dim, hint):
    """Few of many places hold a page, a block's list is refilled, and lengths are past the hint."""
    g, H, R = torch.Generator().manual_seed(hint), 3, 310
    lens = [[3000, 0, 70, 1, 64, 500][int(x)] for x in torch.randint(0, 6, (R,), generator=g)]
    starts = [[0, 64, 65, 2999][int(x)] for x in torch.randint(0, 4, (R,), generator=g)]
    pages = sum(ref.pages_of(n) for n in lens) + 1
    pools = ref.Pools(pages, H, dim, kv, "head")
    table = torch.full((R, 47), -1, dtype=torch.int32)
    perm, at = torch.randperm(pages, generator=g).to(torch.int32), 0
    for r, n in enumerate(lens):
        m = ref.pages_of(n)
        table[r, :m] = perm[at:at + m]
        at += m
        t = torch.arange(n)
        if n:
            x = torch.randn((n, H, dim), generator=g).to(ref.TYPES["fp16" if kv == "fp16" else "bf16"])
            pools.put(table[r].long()[t // PAGE], t % PAGE, x, x)
    bounds, unit = torch.full((pages, H, 2, dim), 77, dtype=torch.int8), torch.full((pages, H), -1.0)
    got, got_unit, status = bounds.cuda(), unit.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    k, _, ks, _ = pools.cuda()
    lib.block_bounds(k, table.cuda(), int32(starts), int32(lens), hint, got, got_unit, k_scale=ks, dev_status=status)
    touched = torch.zeros(pages, dtype=torch.bool)
    for r, n in enumerate(lens):
        for b in range(starts[r] // PAGE, ref.pages_of(n)) if starts[r] < n else ():
            page = int(table[r, b])
            touched[page] = True
            if (r + b) % 9 == 0 or b == ref.pages_of(n) - 1:
                t = torch.arange(b * PAGE, min(n, (b + 1) * PAGE))
                keys, _ = pools.get(torch.full_like(t, page), t % PAGE)
                for h in range(H):
                    box, scale = ref.box(keys[:, h])
                    assert torch.equal(got[page, h].cpu(), box) and float(got_unit[page, h]) == float(scale), (r, b, h)
    assert int(status) == 0
    assert torch.equal((got_unit.cpu() > 0).all(1), touched) and (got.cpu()[~touched] == 77).all()
