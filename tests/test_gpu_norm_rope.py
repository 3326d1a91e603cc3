"""Per-head norm + rotation on the GPU against a 64-bit reference."""
import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def tolerance(want, dtype):
    """Half a step of the type at the value, and fp32 arithmetic (sums of up to 256 terms, the
    reciprocal root, two products of the rotation) at the row's size."""
    row = want.abs().amax(-1, keepdim=True)
    return torch.finfo(dtype).eps / 2 * want.abs() * 1.001 + 2.0 ** -19 * row + 2.0 ** -25


def check(got, want, dtype):
    d = (got.double().cpu() - want).abs()
    assert torch.isfinite(got.float()).all()
    assert (d <= tolerance(want, dtype)).all(), float((d - tolerance(want, dtype)).max())


def run(T, Hq, Hk, D, rot, offset, inter, kind, dtype, seed, affine=True, in_place=False, extra=0):
    g = torch.Generator().manual_seed(seed)
    x = (3 * torch.randn((T, Hq + Hk + extra, D), generator=g)).to(dtype)
    w = [1 + 0.3 * torch.randn(D, generator=g) if affine else None for _ in range(2)]
    b = [0.3 * torch.randn(D, generator=g) if affine else None for _ in range(2)]
    pos = torch.randint(0, 4096, (T,), generator=g, dtype=torch.int32) if rot else None
    table = lib.rope_table(4096, rot) if rot else None
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    xd = x.cuda()
    q, k = xd[:, :Hq], xd[:, Hq:Hq + Hk]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dict(q_out=q, k_out=k) if in_place else {}
    yq, yk = lib.qk_norm_rope(q, k, dev(pos), table, rot_offset=offset, interleaved=inter, norm=kind,
                              q_weight=dev(w[0]), k_weight=dev(w[1]), q_bias=dev(b[0]),
                              k_bias=dev(b[1]), eps=1e-6, dev_status=status, **out)
    torch.cuda.synchronize()
    assert int(status) == 0
    for got, src, i in ((yq, x[:, :Hq], 0), (yk, x[:, Hq:Hq + Hk], 1)):
        check(got, ref.norm_rope(src, kind, w[i], b[i], 1e-6, pos, rot, offset, inter), dtype)
    if extra:
        assert torch.equal(xd[:, Hq + Hk:].cpu(), x[:, Hq + Hk:])      # neighbours untouched


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("kind", [lib.NORM_NONE, lib.NORM_RMS, lib.NORM_LAYER])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot,offset", [(128, 64, 0), (128, 64, 64), (192, 64, 128), (64, 64, 0),
                                          (256, 256, 0), (72, 16, 56)])
def test_types_and_layouts(dtype, kind, inter, D, rot, offset):
    run(7, 5, 2, D, rot, offset, inter, kind, TYPES[dtype], seed=D + rot + kind, extra=1)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 0), (1, 64, 1), (3, 6, 3), (0, 4, 1), (257, 3, 1), (2, 0, 5)])
def test_sizes(T, Hq, Hk):
    run(T, Hq, Hk, 128, 64, 0, False, lib.NORM_LAYER, torch.bfloat16, seed=T + Hq)


def test_smallest_and_plain_dims():
    run(5, 3, 1, 8, 8, 0, True, lib.NORM_RMS, torch.float32, seed=1)
    run(5, 3, 1, 128, 0, 0, False, lib.NORM_RMS, torch.bfloat16, seed=2)          # no rotation
    run(5, 3, 1, 128, 64, 0, False, lib.NORM_RMS, torch.bfloat16, seed=3, affine=False)


def test_in_place():
    run(33, 9, 2, 128, 64, 64, False, lib.NORM_RMS, torch.bfloat16, seed=4, in_place=True)


def test_layer_norm_far_from_zero():
    """A mean far larger than the spread: the variance is taken about the mean."""
    g = torch.Generator().manual_seed(5)
    x = (1000 + torch.randn((16, 2, 128), generator=g)).float()
    y, _ = lib.qk_norm_rope(x.cuda(), None, norm=lib.NORM_LAYER)
    want = ref.norm(x.double(), 2, None, None, 1e-6)
    # the mean's fp32 rounding (a few 2^-24 of 1000) over a spread of 1
    assert (y.double().cpu() - want).abs().max() <= 1000 * 2.0 ** -21 + 2.0 ** -19 * 4


def test_zero_rows_and_non_finite():
    x = torch.zeros((2, 3, 128), dtype=torch.bfloat16, device="cuda")
    x[1, 0, 5] = float("inf")
    x[1, 1, 5] = float("nan")
    y, _ = lib.qk_norm_rope(x, None, norm=lib.NORM_RMS)
    assert (y[0] == 0).all() and (y[1, 2] == 0).all()
    assert torch.isnan(y[1, 0, 5]) and torch.isnan(y[1, 1]).all()


def test_positions_outside_the_table():
    x = torch.randn((4, 3, 128), device="cuda").to(torch.bfloat16)
    table = lib.rope_table(16, 64)
    pos = torch.tensor([3, -1, 16, 15], dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, k = lib.qk_norm_rope(x[:, :2], x[:, 2:], pos, table, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 8
    for out in (y, k):
        assert torch.isnan(out[1:3]).all() and torch.isfinite(out[[0, 3]]).all()


def test_strided_heads_and_other_stream():
    """Heads-major input through strides, on a stream of its own."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn((4, 11, 128), generator=g).to(torch.bfloat16)       # [heads, tokens, D]
    s = torch.cuda.Stream()
    xd = x.cuda()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y, _ = lib.qk_norm_rope(xd.transpose(0, 1), None)
    s.synchronize()
    check(y, ref.norm(x.transpose(0, 1).double(), 1, None, None, 1e-6), torch.bfloat16)
