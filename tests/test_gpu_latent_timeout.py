"""Latent attention when a wait runs out, without a GPU fault.

A test-only build of the library (compiled here into a temporary directory, never shipped) leaves
the first tile of every CTA undelivered and shortens every wait bound to ~10 ms.  The kernel must
report DSA_ERR_TIMEOUT, write NaN to every row that has tokens and zeros to those that have none,
give its tensor memory back and return -- after which the context is still usable.
"""
import ctypes

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref
from tests.test_gpu_latent_attention import Case
from tests.test_gpu_timeout import _build_variant

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def variant(tmp_path_factory):
    L = _build_variant(str(tmp_path_factory.mktemp("timeout")))
    vp, ll, ci, cf = ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_float
    L.dsa_latent_attention.restype = ci
    L.dsa_latent_attention.argtypes = [vp, ll, ll, vp, ll, ll, ci, ci, ci, ci, cf, vp, ll, ci, ci, ci, vp,
                                       ll, ci, vp, vp, ll, ci, vp, ll, ll, vp, vp, ll, vp, vp]
    return L


@pytest.mark.parametrize("kv", [lib.KV_FP8_E4M3, lib.KV_BF16])
@pytest.mark.parametrize("lens", [[40], [1000], [300, 0, 20000, 64]])
def test_wait_that_runs_out(variant, kv, lens):
    H = 24
    c = Case(lens, H, kv, seed=31)
    q, pool, table, seqlens = c.q.cuda(), c.pool.cuda(), c.table.cuda(), c.seqlens.cuda()
    out = torch.full((c.R, H, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.R, H), 3.0, device="cuda")
    ws = torch.empty(lib.dsa_latent_attention_workspace(), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    st = variant.dsa_latent_attention(
        q.data_ptr(), q.stride(0), q.stride(1), q.data_ptr() + 1024, q.stride(0), q.stride(1), c.R, H,
        512, 64, c.scale, pool.data_ptr(), pool.stride(0), pool.shape[0], kv, 64, table.data_ptr(),
        table.stride(0), table.shape[1], seqlens.data_ptr(), None, 0, 0, out.data_ptr(), out.stride(0),
        out.stride(1), lse.data_ptr(), ws.data_ptr(), ws.numel(), status.data_ptr(),
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()                      # returns: the kernel did not hang
    assert int(status) == 5                       # DSA_ERR_TIMEOUT
    for r, n in enumerate(lens):
        if n:
            assert torch.isnan(out[r].float()).all() and torch.isnan(lse[r]).all()
        else:
            assert (out[r] == 0).all() and torch.isneginf(lse[r]).all()
    c.run().check()                               # the product library, in the same context
