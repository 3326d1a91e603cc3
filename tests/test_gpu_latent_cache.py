"""The latent cache's store and load on the GPU."""
import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

KVS = [lib.KV_FP8_E4M3, lib.KV_BF16]


def status_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def inputs(n, seed, magnitude=1.0):
    g = torch.Generator().manual_seed(seed)
    x = magnitude * torch.randn((n, 576), generator=g) * torch.exp(torch.randn((n, 1), generator=g))
    return x.to(torch.bfloat16), g


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("n", [1, 9, 200])
@pytest.mark.parametrize("magnitude", [1.0, 1e-30, 1e30])
def test_store_is_exact_without_norm(kv, n, magnitude):
    x, g = inputs(n, n, magnitude)
    if n > 8:
        x[2, 128:256] = 0                                   # a group of zeros
        x[3, 0] = float("inf")
        x[4, 1] = float("nan")
        x[5, :128] = -0.0
        x[6, 0:128] = 448.0                                 # exactly the largest code
        x[7, 0:128] = 450.0                                 # just past it
    pages = n // 64 + 3
    slots = torch.randperm(pages * 64, generator=g)[:n].to(torch.int32)
    if n > 8:
        slots[8] = -1                                       # a padding token
    pool = torch.full((pages, ref.PAGE_BYTES[kv] + 64), 0x55, dtype=torch.uint8)
    want = pool.clone()
    keep = slots >= 0
    page, slot = slots[keep].long() // 64, slots[keep].long() % 64
    latent, rope, scale = ref.page_views(want, kv)
    rope[page, slot] = x[keep, 512:]
    if kv == lib.KV_BF16:
        latent[page, slot] = x[keep, :512]
    else:
        codes, s = ref.quantise(x[keep, :512].double())
        latent[page, slot] = codes
        scale[page, slot] = s
    # views of a sliced pool are copies where the slice is not contiguous: write them back
    if kv == lib.KV_BF16:
        want[:, :73728] = torch.cat([latent, rope], -1).contiguous().view(torch.uint8).view(pages, -1)
    else:
        want[:, :32768] = latent.reshape(pages, -1)
        want[:, 32768:40960] = rope.contiguous().view(torch.uint8).view(pages, -1)
        want[:, 40960:41984] = scale.contiguous().view(torch.uint8).view(pages, -1)
    dev, st = pool.cuda(), status_word()
    xd = x.cuda()
    lib.latent_store(xd[:, :512], xd[:, 512:], slots.cuda(), dev, kv, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    got = dev.cpu()
    if n > 8 and kv == lib.KV_BF16:
        # a NaN's payload may change: compare it as NaN
        i = int(slots[4])
        a = got[i // 64, (i % 64) * 1152 + 2:(i % 64) * 1152 + 4].clone().view(torch.bfloat16)
        assert torch.isnan(a).all()
        got[i // 64, (i % 64) * 1152 + 2:(i % 64) * 1152 + 4] = 0
        want[i // 64, (i % 64) * 1152 + 2:(i % 64) * 1152 + 4] = 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("inter", [False, True])
def test_store_with_norm_and_rotation(kv, inter):
    n = 130
    x, g = inputs(n, 3)
    w = 1 + 0.2 * torch.randn(512, generator=g)
    pos = torch.randint(0, 8192, (n,), generator=g, dtype=torch.int32)
    pool = torch.zeros((5, ref.PAGE_BYTES[kv]), dtype=torch.uint8, device="cuda")
    slots = torch.randperm(5 * 64, generator=g)[:n].to(torch.int32)
    xd, st = x.cuda(), status_word()
    lib.latent_store(xd[:, :512], xd[:, 512:], slots.cuda(), pool, kv, norm_weight=w.cuda(), eps=1e-6,
                     positions=pos.cuda(), rope_table=lib.rope_table(8192, 64), interleaved=inter,
                     dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    c = ref.norm(x[:, :512].double(), 1, w, None, 1e-6)
    r = ref.rotate(x[:, 512:].double(), ref.angles(pos, 64), inter)
    host = pool.cpu()
    got = ref.tokens(host, kv, slots.long() // 64, slots.long() % 64)
    half = torch.finfo(torch.bfloat16).eps / 2
    arith = 2.0 ** -19                                      # fp32 sums, root and products
    tol = half * r.abs() + arith * r.abs().amax(-1, keepdim=True)
    assert ((got[:, 512:] - r).abs() <= tol).all()
    if kv == lib.KV_BF16:
        tol = half * c.abs() + arith * c.abs()
    else:
        s = ref.page_views(host, kv)[2][slots.long() // 64, slots.long() % 64].double()
        top = c.view(n, 4, 128).abs().amax(-1)
        assert (torch.exp2(torch.log2(s).round()) == s).all()
        assert (top <= 448 * s * (1 + 2.0 ** -20)).all() and (top > 224 * s * (1 - 2.0 ** -20)).all()
        s = s.repeat_interleave(128, -1)
        # half a step of e4m3: 2^-4 of the value, 2^-10 of the scale below 2^-6 of it
        tol = torch.maximum(2.0 ** -4 * c.abs(), 2.0 ** -10 * s) + arith * c.abs()
    assert ((got[:, :512] - c).abs() <= tol).all()


@pytest.mark.parametrize("kv", KVS)
def test_store_reports_bad_slots_and_positions(kv):
    x, _ = inputs(4, 5)
    x = x.cuda()
    pool = torch.zeros((2, ref.PAGE_BYTES[kv]), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([0, 128, 64, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    st = status_word()
    lib.latent_store(x[:, :512], x[:, 512:], slots, pool, kv, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 6
    st = status_word()
    lib.latent_store(x[:2, :512], x[:2, 512:], slots[:1].repeat(2) + torch.arange(2, device="cuda", dtype=torch.int32),
                     pool, kv, positions=torch.tensor([9, 3], dtype=torch.int32, device="cuda"),
                     rope_table=lib.rope_table(9, 64), dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 8
    t = ref.tokens(pool.cpu(), kv, torch.tensor([0, 0]), torch.tensor([0, 1]))
    assert torch.isnan(t[0, 512:]).all() and torch.isfinite(t[0, :512]).all() and torch.isfinite(t[1]).all()


@pytest.mark.parametrize("kv", KVS)
@pytest.mark.parametrize("lens,starts", [([1], [0]), ([65], [3]), ([0, 5, 0, 0, 130, 64, 0], None),
                                         ([3, 100, 1], [60, 64, 127]), ([1] * 70, None)])
def test_load_ragged(kv, lens, starts):
    g = torch.Generator().manual_seed(len(lens))
    B = len(lens)
    W = max(1, max((n + (starts[i] if starts else 0) + 63) // 64 for i, n in enumerate(lens)))
    pool = ref.random_pool(B * W + 2, kv, g, ref.PAGE_BYTES[kv] + 128)
    table = torch.randperm(B * W + 2, generator=g)[:B * W].to(torch.int32).view(B, W)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    n = int(cu[-1])
    out = torch.full((n + 3, 600), 7.0, dtype=torch.bfloat16, device="cuda")
    st = status_word()
    lib.latent_load(pool.cuda(), kv, table.cuda(), cu.cuda(), n + 3,
                    starts=None if starts is None else torch.tensor(starts, dtype=torch.int32).cuda(),
                    out=out[:, :576], dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    got = out.cpu()
    assert (got[:, 576:] == 7).all() and (got[n:, :576] == 0).all()
    want = []
    for b, m in enumerate(lens):
        t = torch.arange(m) + (starts[b] if starts else 0)
        want.append(ref.tokens(pool, kv, table[b].long()[t // 64], t % 64))
    # the pool's scales are powers of two: reading back is exact
    assert torch.equal(got[:n, :576].double(), torch.cat(want))


@pytest.mark.parametrize("kv", KVS)
def test_load_reports_bad_pages_and_positions(kv):
    g = torch.Generator().manual_seed(9)
    pool = ref.random_pool(3, kv, g)
    table = torch.tensor([[0, 7], [-1, 2]], dtype=torch.int32)
    cu = torch.tensor([0, 70, 140], dtype=torch.int32)
    st = status_word()
    out = lib.latent_load(pool.cuda(), kv, table.cuda(), cu.cuda(), 140, dev_status=st).cpu()
    assert int(st) == 6
    assert torch.isfinite(out[:64]).all() and torch.isnan(out[64:70]).all()
    assert torch.isnan(out[70:134]).all() and torch.isfinite(out[134:]).all()
    st = status_word()
    starts = torch.tensor([0, -1], dtype=torch.int32).cuda()
    out = lib.latent_load(pool.cuda(), kv, torch.zeros((2, 1), dtype=torch.int32).cuda(),
                          torch.tensor([0, 65, 67], dtype=torch.int32).cuda(), 67, starts=starts,
                          dev_status=st).cpu()
    assert int(st) == 7
    assert torch.isfinite(out[:64]).all() and torch.isnan(out[64:66]).all() and torch.isfinite(out[66]).all()


@pytest.mark.parametrize("kv", KVS)
def test_page_past_4_gib(kv):
    """A pool whose last page lies past 2^32 bytes."""
    pages = 2 ** 32 // ref.PAGE_BYTES[kv] + 2
    pool = torch.empty((pages, ref.PAGE_BYTES[kv]), dtype=torch.uint8, device="cuda")
    x, _ = inputs(2, 8)
    xd = x.cuda()
    slots = torch.tensor([(pages - 1) * 64 + 63, 5], dtype=torch.int32, device="cuda")
    lib.latent_store(xd[:, :512], xd[:, 512:], slots, pool, kv)
    table = torch.tensor([[pages - 1], [0]], dtype=torch.int32, device="cuda")
    out = lib.latent_load(pool, kv, table, torch.tensor([0, 1, 2], dtype=torch.int32).cuda(), 2,
                          starts=torch.tensor([63, 5], dtype=torch.int32).cuda()).cpu()
    if kv == lib.KV_BF16:
        want = x.double()
    else:
        codes, s = ref.quantise(x[:, :512].double())
        c = codes.view(torch.float8_e4m3fn).float().double() * s.double().repeat_interleave(128, -1)
        want = torch.cat([c, x[:, 512:].double()], -1)
    assert torch.equal(out.double(), want)
