"""Host-side argument checks of the calls around the sparse attention (no GPU: every call here is
refused, or has nothing to launch, before any device work)."""
import os
import shutil

import pytest

from sparse_attention_paged_gb300 import _native

pytestmark = pytest.mark.skipif(shutil.which(_native.NVCC) is None and
                                not os.path.exists(_native.LIB_PATH),
                                reason="nvcc not available and library not built")

A = 0x10000          # a fake, aligned device address
OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3


def norm_rope(**kw):
    import sparse_attention_paged_gb300 as s
    args = dict(q=A, q_token_stride=8192, q_head_stride=128, Hq=64, k=A, k_token_stride=128,
                k_head_stride=128, Hk=1, T=4, D=128, dtype=s.BF16, norm=s.NORM_RMS, q_weight=A,
                k_weight=A, q_bias=None, k_bias=None, eps=1e-6, positions=A, rope_table=A,
                max_pos=64, rot_dims=64, rot_offset=0, interleaved=0, q_out=A, qo_token_stride=8192,
                qo_head_stride=128, k_out=A, ko_token_stride=128, ko_head_stride=128, stream=0)
    args.update(kw)
    return s.dsa_qk_norm_rope(**args)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(T=0)), (OK, dict(Hq=0, Hk=0)), (OK, dict(T=0, q=None, k=None)),
    (INVALID, dict(T=-1)), (INVALID, dict(Hq=-1)), (INVALID, dict(dtype=3)), (INVALID, dict(norm=4)),
    (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("nan"))), (INVALID, dict(q=None)),
    (INVALID, dict(k_out=None)), (INVALID, dict(rope_table=None)), (INVALID, dict(max_pos=0)),
    (INVALID, dict(rot_dims=0)), (INVALID, dict(rot_dims=144)), (INVALID, dict(rot_offset=72)),
    (INVALID, dict(rot_offset=-8)),
    (UNSUPPORTED, dict(D=0)), (UNSUPPORTED, dict(D=100)), (UNSUPPORTED, dict(D=264)),
    (UNSUPPORTED, dict(rot_dims=24)), (UNSUPPORTED, dict(rot_offset=4)),
    (UNSUPPORTED, dict(rot_dims=20, interleaved=1)), (UNSUPPORTED, dict(T=2 ** 31 - 1)),
    (MISALIGNED, dict(q=A + 8)), (MISALIGNED, dict(k_out=A + 2)), (MISALIGNED, dict(q_head_stride=132)),
    (MISALIGNED, dict(ko_token_stride=4)), (MISALIGNED, dict(rope_table=A + 4)),
    (MISALIGNED, dict(q_weight=A + 2)), (MISALIGNED, dict(positions=A + 1)),
    (MISALIGNED, dict(dtype=2, q_token_stride=2)),
])
def test_norm_rope_refusals(want, kw):
    assert norm_rope(**kw) == want


def store(**kw):
    import sparse_attention_paged_gb300 as s
    args = dict(latent=A, latent_stride=576, rope=A, rope_stride=576, n=4, latent_dim=512, rope_dim=64,
                norm_weight=A, eps=1e-6, positions=A, rope_table=A, max_pos=8, interleaved=1,
                slot_mapping=A, cache=A, page_stride_bytes=41984, num_pages=2, kv_dtype=0,
                page_size=64, stream=0)
    args.update(kw)
    return s.dsa_latent_store(**args)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=0)), (OK, dict(n=0, latent=None, rope=None, slot_mapping=None)),
    (INVALID, dict(n=-1)), (INVALID, dict(eps=-1e-6)), (INVALID, dict(latent=None)),
    (INVALID, dict(rope=None)), (INVALID, dict(slot_mapping=None)), (INVALID, dict(cache=None)),
    (INVALID, dict(num_pages=0)), (INVALID, dict(kv_dtype=2)), (INVALID, dict(page_stride_bytes=41968)),
    (INVALID, dict(kv_dtype=1, page_stride_bytes=73712)), (INVALID, dict(rope_table=None)),
    (INVALID, dict(max_pos=0)),
    (UNSUPPORTED, dict(latent_dim=256)), (UNSUPPORTED, dict(rope_dim=32)), (UNSUPPORTED, dict(page_size=16)),
    (MISALIGNED, dict(latent=A + 8)), (MISALIGNED, dict(latent_stride=516)), (MISALIGNED, dict(rope=A + 2)),
    (MISALIGNED, dict(rope_stride=65)), (MISALIGNED, dict(cache=A + 4)),
    (MISALIGNED, dict(page_stride_bytes=41992)), (MISALIGNED, dict(norm_weight=A + 4)),
    (MISALIGNED, dict(slot_mapping=A + 2)),
])
def test_store_refusals(want, kw):
    assert store(**kw) == want


def load(**kw):
    import sparse_attention_paged_gb300 as s
    args = dict(cache=A, page_stride_bytes=73728, num_pages=2, kv_dtype=1, page_size=64, block_table=A,
                bt_stride=4, W=4, starts=None, cu_rows=A, n_req=3, n=10, latent_dim=512, rope_dim=64,
                out=A, out_stride=576, stream=0)
    args.update(kw)
    return s.dsa_latent_load(**args)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(n=0)), (OK, dict(n=0, n_req=0, out=None, cu_rows=None)),
    (INVALID, dict(n=-1)), (INVALID, dict(n_req=-1)), (INVALID, dict(n_req=0)), (INVALID, dict(W=0)),
    (INVALID, dict(bt_stride=3)), (INVALID, dict(bt_stride=-1)), (INVALID, dict(block_table=None)),
    (INVALID, dict(cu_rows=None)), (INVALID, dict(out=None)), (INVALID, dict(out_stride=568)),
    (INVALID, dict(cache=None)), (INVALID, dict(num_pages=-1)),
    (UNSUPPORTED, dict(latent_dim=511)), (UNSUPPORTED, dict(page_size=32)),
    (MISALIGNED, dict(out=A + 8)), (MISALIGNED, dict(out_stride=580)), (MISALIGNED, dict(cu_rows=A + 1)),
    (MISALIGNED, dict(starts=A + 2)), (MISALIGNED, dict(cache=A + 8)),
])
def test_load_refusals(want, kw):
    assert load(**kw) == want


def attention(**kw):
    import sparse_attention_paged_gb300 as s
    args = dict(q_latent=A, ql_row_stride=64 * 512, ql_head_stride=512, q_rope=A, qr_row_stride=64 * 64,
                qr_head_stride=64, rows=2, H=64, latent_dim=512, rope_dim=64, scale=0.1, cache=A,
                page_stride_bytes=41984, num_pages=8, kv_dtype=0, page_size=64, block_table=A,
                bt_stride=4, W=4, seqlens=A, idx=A, idx_stride=128, k=128, out=A,
                out_row_stride=64 * 512, out_head_stride=512, lse=A, workspace=A,
                workspace_floats=1 << 40, stream=0)
    args.update(kw)
    return s.dsa_latent_attention(**args)


@pytest.mark.parametrize("want,kw", [
    (OK, dict(rows=0)), (OK, dict(rows=0, q_latent=None, workspace=None, workspace_floats=0)),
    (INVALID, dict(rows=-1)), (INVALID, dict(H=0)), (INVALID, dict(W=0)),
    (INVALID, dict(scale=float("inf"))), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(bt_stride=2)), (INVALID, dict(bt_stride=-4)), (INVALID, dict(k=0)),
    (INVALID, dict(idx_stride=127)), (INVALID, dict(q_latent=None)), (INVALID, dict(q_rope=None)),
    (INVALID, dict(block_table=None)), (INVALID, dict(seqlens=None)), (INVALID, dict(out=None)),
    (INVALID, dict(workspace=None)), (INVALID, dict(cache=None)), (INVALID, dict(kv_dtype=-1)),
    (INVALID, dict(page_stride_bytes=8448)),
    (UNSUPPORTED, dict(H=129)), (UNSUPPORTED, dict(latent_dim=128)), (UNSUPPORTED, dict(rope_dim=0)),
    (UNSUPPORTED, dict(page_size=1)), (UNSUPPORTED, dict(rows=2 ** 30, idx=None)),
    (UNSUPPORTED, dict(rows=1, W=2 ** 25, bt_stride=0)),
    (MISALIGNED, dict(q_latent=A + 8)), (MISALIGNED, dict(q_rope=A + 2)),
    (MISALIGNED, dict(ql_head_stride=516)), (MISALIGNED, dict(qr_row_stride=4)),
    (MISALIGNED, dict(out=A + 8)), (MISALIGNED, dict(out_head_stride=514)),
    (MISALIGNED, dict(workspace=A + 8)), (MISALIGNED, dict(seqlens=A + 2)),
    (MISALIGNED, dict(idx=A + 1)), (MISALIGNED, dict(lse=A + 2)),
])
def test_attention_refusals(want, kw):
    assert attention(**kw) == want


def test_attention_without_a_device_or_workspace():
    """A valid call that no device can take, or whose workspace is too small, launches nothing."""
    import torch
    import sparse_attention_paged_gb300 as s
    if torch.cuda.is_available():
        assert s.dsa_latent_attention_workspace() > 0
        assert attention(workspace_floats=s.dsa_latent_attention_workspace() - 1) == INVALID
    else:
        assert s.dsa_latent_attention_workspace() == -1
        assert attention() == 4


def test_tensor_calls_refuse_wrong_tensors():
    import torch
    import sparse_attention_paged_gb300 as s
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="table"):
        s.qk_norm_rope(q, None, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="positions"):
        s.qk_norm_rope(q, None, torch.zeros(3, dtype=torch.int32), torch.zeros((4, 64)))
    with pytest.raises(ValueError, match="q_weight"):
        s.qk_norm_rope(q, None, q_weight=torch.zeros(64))
    with pytest.raises(ValueError, match="CUDA"):
        s.qk_norm_rope(q, None)
    with pytest.raises(ValueError, match="expected"):
        s.qk_norm_rope(q.double(), None)
    pool = torch.zeros((2, 41984), dtype=torch.uint8)
    lat, rope = torch.zeros((3, 512), dtype=torch.bfloat16), torch.zeros((3, 64), dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="shorter"):
        s.latent_store(lat, rope, slots, pool, s.KV_BF16)
    with pytest.raises(ValueError, match="slot_mapping"):
        s.latent_store(lat, rope, slots.long(), pool, s.KV_FP8_E4M3)
    with pytest.raises(ValueError, match="latent"):
        s.latent_store(lat.float(), rope, slots, pool, s.KV_FP8_E4M3)
    bt = torch.zeros((2, 4), dtype=torch.int32)
    ql, qr = torch.zeros((3, 8, 512), dtype=torch.bfloat16), torch.zeros((3, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="one row"):
        s.latent_attention(ql, qr, pool, s.KV_FP8_E4M3, bt, slots, 0.1, out=ql, workspace=torch.zeros(1))
    with pytest.raises(ValueError, match="idx"):
        s.latent_attention(ql, qr, pool, s.KV_FP8_E4M3, bt[:1], slots, 0.1, idx=bt)
    with pytest.raises(ValueError, match="q_rope"):
        s.latent_attention(ql, qr[:, :4], pool, s.KV_FP8_E4M3, bt[:1], slots, 0.1)
