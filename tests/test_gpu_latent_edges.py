"""The latent cache's operators at the edges: large stores, pools past 4 GiB, unusual scales and
query sizes, captured calls, gaps between pages."""
import math

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref
from tests.test_gpu_latent_attention import Case

pytestmark = pytest.mark.gpu

KVS = [lib.KV_FP8_E4M3, lib.KV_BF16]


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("n", [4095, 4096, 4097])
@pytest.mark.parametrize("norm", [False, True])
def test_large_store_is_small_stores(kv, n, norm):
    """From 4,096 tokens on a warp stores two: the same bytes as in calls of 1,000."""
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn((n, 576), generator=g, device="cuda").to(torch.bfloat16)
    pages = n // 64 + 2
    slots = torch.randperm(pages * 64, generator=g, device="cuda")[:n].to(torch.int32)
    slots[5] = slots[6] = slots[100] = slots[n - 1] = -1          # padding: either token of a warp, or both
    slots[7], slots[20] = pages * 64, 2 ** 31 - 1                 # past the pool: reported and skipped
    more = {}
    pos = None
    if norm:
        pos = torch.randint(0, 500, (n,), generator=g, device="cuda", dtype=torch.int32)
        pos[31] = -3                                              # its rotated part: NaN, reported
        more = {"norm_weight": 1 + 0.2 * torch.randn(512, generator=g, device="cuda"),
                "rope_table": lib.rope_table(500, 64)}
    pools = [torch.full((pages, lib.LATENT_PAGE_BYTES[kv]), 0x55, dtype=torch.uint8, device="cuda")
             for _ in range(2)]
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    lib.latent_store(x[:, :512], x[:, 512:], slots, pools[0], kv, positions=pos, dev_status=st[:1], **more)
    for i in range(0, n, 1000):
        j = min(i + 1000, n)
        lib.latent_store(x[i:j, :512], x[i:j, 512:], slots[i:j], pools[1], kv,
                         positions=None if pos is None else pos[i:j].clone(), dev_status=st[1:], **more)
    torch.cuda.synchronize()
    assert int(st[0]) != 0 and int(st[1]) != 0
    assert torch.equal(pools[0], pools[1])


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("k", [0, 190])
def test_attention_over_pages_past_4_gib(kv, k):
    """The same pages at the end of a pool of 5 GiB give the same bits."""
    c = Case([300, 64, 1], 37, kv, k=k, seed=8).run().check()
    small = c.pool
    pages = 5 * 2 ** 30 // ref.PAGE_BYTES[kv]
    big = torch.empty((pages, ref.PAGE_BYTES[kv]), dtype=torch.uint8, device="cuda")
    big[-len(small):] = small.cuda()
    table = torch.where(c.table < len(small), c.table + (pages - len(small)), c.table)
    q = c.q.cuda()
    lse = torch.empty_like(c.lse)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = lib.latent_attention(q[..., :512], q[..., 512:], big, kv, table.cuda(), c.seqlens.cuda(), c.scale,
                               idx=None if c.idx is None else c.idx.cuda(), lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    assert torch.equal(out, c.out) and torch.equal(lse, c.lse)


def test_scales_that_are_no_powers_of_two():
    """Another writer's scales: ratio and product are rounded, 2^-11 of a value each."""
    c = Case([200, 129], 20, lib.KV_FP8_E4M3, seed=9)
    g = torch.Generator().manual_seed(1)
    scale = ref.page_views(c.pool, c.kv)[2]
    c.pool[:, 40960:41984] = (scale * (0.5 + torch.rand(scale.shape, generator=g))).contiguous() \
        .view(torch.uint8).view(len(c.pool), -1)
    c.run()
    assert int(c.status) == 0
    off = 2.0 ** -10 * (1 + 2.0 ** -10)
    for r in range(c.R):
        t = torch.arange(c.lens[r])
        kv = ref.tokens(c.pool, c.kv, c.table[r].long()[t // 64], t % 64)
        q = c.q[r].double()
        want, lse, bound, lse_bound = ref.attention_row(q, kv, c.scale)
        score = off * abs(c.scale) * (q[:, :512].abs() @ kv[:, :512].abs().T).amax(-1)
        size = torch.softmax(c.scale * (q @ kv.T), -1) @ kv[:, :512].abs()
        more = (off + torch.expm1(2 * score)[:, None]) * size * 1.02
        assert ((c.out[r].double().cpu() - want).abs() <= bound + more).all()
        assert ((c.lse[r].double().cpu() - lse).abs() <= lse_bound + score).all()


@pytest.mark.parametrize("size", [1e-30, 1e-4, 300.0])
def test_query_sizes(size):
    """fp8 queries are brought into fp16's range by a power of two per head, each its own."""
    c = Case([150, 70], 9, lib.KV_FP8_E4M3, seed=10)
    c.q[:, ::2] = (c.q[:, ::2].float() * size).to(torch.bfloat16)
    c.run().check()


@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_bad_scale_stays_in_its_row(value):
    c = Case([100, 100, 100], 5, lib.KV_FP8_E4M3, seed=11)
    page = int(c.table[1, 0])
    c.pool[page, 40960 + 16 * 7:40960 + 16 * 7 + 4] = torch.tensor([value], dtype=torch.float32).view(torch.uint8)
    c.run()
    assert torch.isnan(c.out[1].float()).any() and torch.isnan(c.lse[1]).all()
    c.check(rows=[0, 2])


def test_zero_scales():
    """A group of zeros under a zero scale, and a token of nothing else."""
    c = Case([130], 5, lib.KV_FP8_E4M3, seed=12)
    p0 = int(c.table[0, 0])
    view = c.pool[p0, 40960:41984].view(torch.float32).view(64, 4)
    view[3, 1] = 0.0
    view[9] = 0.0
    c.run().check()


@pytest.mark.parametrize("kv", KVS)
def test_load_with_gaps_between_pages(kv):
    g = torch.Generator().manual_seed(4)
    pool = ref.random_pool(4, kv, g, ref.PAGE_BYTES[kv] + 48)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32)
    cu = torch.tensor([0, 150], dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.latent_load(pool.cuda(), kv, table.cuda(), cu.cuda(), 150, dev_status=st)
    t = torch.arange(150)
    want = ref.tokens(pool, kv, table[0].long()[t // 64], t % 64)
    assert int(st) == 0
    assert torch.equal(got.double().cpu(), want)


@pytest.mark.parametrize("kv", KVS)
def test_captured_store_attention_load(kv):
    """A captured step replayed with other tokens in the same buffers."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, pages = 70, 3
    lat, rope = (torch.empty((n, d), dtype=torch.bfloat16, device="cuda") for d in (512, 64))
    pool = torch.zeros((pages, lib.LATENT_PAGE_BYTES[kv]), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[1, 2]], dtype=torch.int32, device="cuda")
    slots = (64 + torch.arange(n, device="cuda")).to(torch.int32)
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    length = torch.tensor([n], dtype=torch.int32, device="cuda")
    q = torch.empty((1, 8, 576), dtype=torch.bfloat16, device="cuda")
    qn = torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    w, pos = torch.ones(128, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    back = torch.empty((n, 576), dtype=torch.bfloat16, device="cuda")
    out, turned = torch.empty((1, 8, 512), dtype=torch.bfloat16, device="cuda"), torch.empty_like(qn)
    work = torch.empty(lib.dsa_latent_attention_workspace(), device="cuda")
    rope_t = lib.rope_table(64, 64)

    def step():
        lib.latent_store(lat, rope, slots, pool, kv)
        lib.qk_norm_rope(qn, None, pos, rope_t, norm=lib.NORM_RMS, q_weight=w, q_out=turned)
        lib.latent_attention(q[..., :512], q[..., 512:], pool, kv, table, length, 0.1, out=out, workspace=work)
        lib.latent_load(pool, kv, table, cu, n, out=back)

    def fill():
        for x in (lat, rope, q, qn):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        pos.fill_(int(torch.randint(0, 64, (1,), generator=g, device="cuda")))

    fill()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        fill()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, back, turned)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, back, turned)):
            assert torch.equal(a, b)
        if kv == lib.KV_BF16:
            assert torch.equal(back, torch.cat([lat, rope], -1))


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("rows,length", [(19, 512), (20, 512), (32, 257), (33, 64), (40, 129), (160, 100), (3, 3201)])
def test_rows_and_lengths_around_the_split(kv, rows, length):
    """Half tiles or whole ones, records by row or by CTA, joins of both kinds."""
    lens = [length + (r % 3) - 1 for r in range(rows)]
    lens[rows // 2] = 0
    Case(lens, 5, kv, seed=rows + length).run().check()


@pytest.mark.parametrize("kv", KVS)
def test_joined_rows_do_not_keep_an_earlier_calls_records(kv):
    """The same workspace for calls whose rows are cut, whole and empty in turn."""
    work = torch.full((lib.dsa_latent_attention_workspace(),), math.nan, device="cuda")
    for lens in ([4000, 4000], [60, 0], [0, 9000], [130] * 30, [0] * 3 + [2000], [70] * 200, [500, 1]):
        Case(lens, 7, kv, seed=len(lens)).run(workspace=work).check()
