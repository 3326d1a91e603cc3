"""The decode step of examples/sparse_decode_step.py: every stage against 64 bits, and its replay."""
import importlib.util
import os

import pytest
import torch

import sparse_attention_paged_gb300 as lib
from tests import latent_ref as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "sparse_decode_step.py")


def example():
    spec = importlib.util.spec_from_file_location("sparse_decode_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def check(s):
    """The step's outputs from its inputs and caches, row by row."""
    assert int(s.status) == 0
    pos = s.positions.cpu()
    table, pool, index_pool = s.block_table.cpu(), s.latent_cache.cpu(), s.index_cache.cpu()
    w = [x.cpu() for x in s.index_norm + s.index_bias + [s.latent_norm]]
    iq = ref.norm_rope(s.index_q.cpu(), 2, w[0], w[2], 1e-6, pos, 64, 0, False)
    ik = ref.norm_rope(s.index_k.cpu(), 2, w[1], w[3], 1e-6, pos, 64, 0, False)
    half = torch.finfo(torch.bfloat16).eps / 2
    for got, want in ((s.index_q_out, iq), (s.index_k_out, ik)):
        assert ((got.double().cpu() - want).abs() <=
                half * want.abs() * 1.001 + 2.0 ** -19 * want.abs().amax(-1, keepdim=True)).all()
    qr = ref.rotate(s.q_rope.cpu().double(), ref.angles(pos, 64)[:, None], True)
    assert ((s.q_rope_out.double().cpu() - qr).abs() <= half * qr.abs() + 2.0 ** -19 * qr.abs().amax(-1, keepdim=True)).all()
    q = torch.cat([s.q_latent, s.q_rope_out], -1).double().cpu()
    idx, out, lse = s.idx.cpu(), s.out.double().cpu(), s.lse.double().cpu()
    iqo, iw = s.index_q_out.double().cpu(), s.index_w.double().cpu()
    for b in range(s.B):
        n = int(pos[b]) + 1
        chosen = idx[b][idx[b] >= 0].long()
        assert len(chosen) == min(n, s.topk) and (chosen < n).all() and (chosen[1:] > chosen[:-1]).all()
        t = torch.arange(n)
        page, slot = table[b].long()[t // 64], t % 64
        # a valid selection of the indexer's logits, within their fp32 and two-term error
        codes = index_pool[:, :8192].view(-1, 64, 128)[page, slot].view(torch.float8_e4m3fn).float().double()
        sc = index_pool[:, 8192:8448].view(torch.float32)[page, slot].double()
        logits = sc * (iw[b][:, None] * torch.relu(iqo[b] @ codes.T)).sum(0)
        if len(chosen) < n:
            rest = torch.ones(n, dtype=torch.bool)
            rest[chosen] = False
            assert logits[chosen].min() >= logits[rest].max() - 2e-3 * logits.abs().max()
        kv = ref.tokens(pool, s.kv, table[b].long()[chosen // 64], chosen % 64)
        want, l64, bound, lse_bound = ref.attention_row(q[b], kv, s.scale)
        assert ((out[b] - want).abs() <= bound).all()
        assert ((lse[b] - l64).abs() <= lse_bound).all()
        # the new token is in the cache
        c = ref.norm(s.latent[b:b + 1].cpu().double(), 1, w[4], None, 1e-6)[0]
        new = ref.tokens(pool, s.kv, page[-1:], slot[-1:])[0, :512]
        assert ((new - c).abs() <= 2.0 ** -4 * c.abs() + 2.0 ** -9 * c.abs().max() / 224).all()


@pytest.mark.parametrize("kv", [lib.KV_FP8_E4M3, lib.KV_BF16])
def test_step_and_replay(kv):
    m = example()
    s = m.SparseDecodeStep(5, 1500, heads=24, topk=128, kv_dtype=kv)
    m.fill(s, [1, 63, 700, 1024, 1400])
    s.run()
    torch.cuda.synchronize()
    check(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for _ in range(2):                                    # two more tokens of every request
        s.positions += 1
        s.latent.copy_(torch.randn_like(s.latent.float()))
        s.q_latent.copy_(torch.randn_like(s.q_latent.float()))
        s.index_q.copy_(torch.randn_like(s.index_q.float()))
        graph.replay()
        torch.cuda.synchronize()
        check(s)
