"""fp8 cache: groups of zeros, whose scale says nothing, and groups of far smaller scales than their
token's largest, as latent_store writes them."""
import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

FP8 = lib.KV_FP8_E4M3


def attend(x, q, scale, idx=None):
    """Stores the tokens x [n, 576], attends over them (q [H, 576]) and holds every element to the
    bounds of a computation with bf16 weights and results."""
    n, pages = len(x), (len(x) + 63) // 64
    pool = torch.zeros((pages, ref.PAGE_BYTES[FP8]), dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)[None]
    t = torch.arange(n, device="cuda")
    slots = (table[0].long()[t // 64] * 64 + t % 64).to(torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    xd, qd = x.cuda(), q.cuda()[None]
    lib.latent_store(xd[:, :512], xd[:, 512:], slots, pool, FP8, dev_status=st)
    lse = torch.empty((1, len(q)), device="cuda")
    out = lib.latent_attention(qd[..., :512], qd[..., 512:], pool, FP8, table,
                               torch.tensor([n], dtype=torch.int32, device="cuda"), scale,
                               idx=None if idx is None else idx.cuda()[None], lse=lse, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == 0
    slots = slots.long().cpu()
    if idx is not None:
        slots = slots[idx.long()]
    tokens = ref.tokens(pool.cpu(), FP8, slots // 64, slots % 64)
    want, lse64, bound, lse_bound = ref.attention_row(q.double(), tokens, scale)
    d = (out[0].double().cpu() - want).abs()
    assert (d <= bound).all(), (float((d / bound.clamp(min=1e-300)).max()), float(d.max()))
    assert ((lse[0].double().cpu() - lse64).abs() <= lse_bound).all()
    return tokens


def inputs(n, H, seed, size, q_size):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, 576), generator=g)
    x[:, :512] *= size
    q = torch.randn((H, 576), generator=g)
    q[:, :512] *= q_size
    return x, q.to(torch.bfloat16)


@pytest.mark.parametrize("n", [70, 300, 5000])
@pytest.mark.parametrize("size", [1e-6, 1e-3, 1.0, 300.0])
def test_zero_groups_beside_others(n, size):
    """Every pattern of zero groups, among them tokens of nothing else; a group of values between
    224 and 448 has scale 1 as well and is no group of zeros."""
    x, q = inputs(n, 12, n, size, 0.05 / size)
    for i in range(n):
        for g in range(4):
            if (i >> g) & 1:
                x[i, g * 128:(g + 1) * 128] = 0.0 if i % 3 else -0.0
    x = x.to(torch.bfloat16)
    tokens = attend(x, q, 0.1)
    assert (tokens[15, :512] == 0).all()


def test_zero_groups_in_a_list():
    x, q = inputs(400, 9, 5, 2e-6, 1e4)
    x[::2, 128:256] = 0
    x[::5, :512] = 0
    g = torch.Generator().manual_seed(6)
    attend(x.to(torch.bfloat16), q, 0.1, idx=torch.randperm(400, generator=g)[:150].to(torch.int32))


def test_one_nonzero_code_in_a_group():
    """A group of scale 1 whose only value is its last one."""
    x, q = inputs(130, 5, 7, 1e-6, 0.01)
    x[:, 384:512] = 0
    x[1::2, 511] = 300.0
    attend(x.to(torch.bfloat16), q, 0.01)


@pytest.mark.parametrize("smaller", [12, 20, 26, 30])
def test_groups_of_far_smaller_scales(smaller):
    """Scales down to 2^-30 of the token's largest.  Below 2^-22 a code is rounded to 2^-32 of the
    largest scale, a quarter of a unit at 2^-30 and for codes below eight only, where the mean
    magnitude of a group is above 60: 2^-8 of it, the bound's share for a rounded weight."""
    x, q = inputs(200, 7, smaller, 1.0, 0.05)
    x[:, 128:256] *= 2.0 ** -smaller
    x[:, 384:512] *= 2.0 ** -(smaller // 2)
    tokens = attend(x.to(torch.bfloat16), q, 0.1)
    assert (tokens[:, 128:256] != 0).any()


@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 100, 2.0 ** 117, 2.0 ** 124])
def test_large_queries(size):
    """Every finite bf16 query has its place in fp16 under its head's power of two."""
    x, q = inputs(150, 6, 3, 1.0, 1.0)
    q = (q.double() * size).to(torch.bfloat16)
    attend(x.to(torch.bfloat16), q, 0.07 / size)


@pytest.mark.parametrize("latent,rotated", [(1e-30, 2.0 ** 30), (1e-37, 1.0), (1e-20, 2.0 ** 100), (0.0, 2.0 ** 120),
                                            (2.0 ** -126, 1e-30), (1.0, 2.0 ** 40)])
def test_query_parts_of_far_sizes(latent, rotated):
    """The head's power of two suits its rotated part too."""
    x, q = inputs(150, 6, 4, 1.0, 1.0)
    q = torch.cat([q[:, :512].double() * latent, q[:, 512:].double() * rotated], -1).to(torch.bfloat16)
    attend(x.to(torch.bfloat16), q, 0.1 / max(rotated, 22 * latent))
