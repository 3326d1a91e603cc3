"""The layer of examples/block_sparse_step.py: prompts and decode steps, every stage against 64 bits,
and the step's replay."""
import importlib.util
import os

import pytest
import torch

from tests import latent_ref
from tests import paged_ref as ref

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "block_sparse_step.py")
HALF = ref.HALF[torch.bfloat16]


def layer_of(*args, **kw):
    spec = importlib.util.spec_from_file_location("block_sparse_step", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m.BlockSparseLayer(*args, **kw)


class Shadow:
    """What every request's tokens are, kept beside the layer on the CPU."""

    def __init__(self, layer, fp8):
        self.layer, self.fp8 = layer, fp8
        self.k = [[] for _ in range(layer.B)]
        self.v = [[] for _ in range(layer.B)]

    def turned(self, x, weight, positions):
        """Norm and rotation in 64 bits, and as bf16 values that the kernel's may be a step off."""
        return latent_ref.norm_rope(x, 1, weight.cpu(), None, 1e-6, positions, self.layer.dim, 0, False)

    def check(self, qkv, counts, q, out, blocks, before):
        """After `counts` new tokens of each request, whose rows were `qkv`."""
        s = self.layer
        assert int(s.status) == 0
        qkv, out, blocks = qkv.cpu(), out.double().cpu(), blocks.cpu()
        table, group = s.block_table.cpu(), s.heads // s.kv_heads
        pools = ref.Pools(1, s.kv_heads, s.dim, "fp8" if self.fp8 else "bf16")
        pools.k, pools.v = s.k_cache.cpu(), s.v_cache.cpu()
        pools.k_scale = s.k_scale.cpu() if self.fp8 else None
        pools.v_scale = s.v_scale.cpu() if self.fp8 else None
        bounds, unit = s.bounds.cpu(), s.bound_scale.cpu()
        held = set()
        row = 0
        for b, n in enumerate(counts):
            total = before[b] + n
            assert int(s.lengths[b]) == total
            pages = table[b, :ref.pages_of(total)].tolist()
            assert len(set(pages)) == len(pages) and not held & set(pages) and min(pages, default=0) >= 0
            held |= set(pages)
            assert (table[b, len(pages):] == -1).all()
            t = torch.arange(total)
            page, slot = table[b].long()[t // 64], t % 64
            k, v = pools.get(page, slot)
            # the new tokens: normed and turned keys, values as they came, to the cache's precision
            x = qkv[row:row + n]
            kx = self.turned(x[:, s.heads:s.heads + s.kv_heads], s.k_norm, t[before[b]:])
            vx = x[:, s.heads + s.kv_heads:].double()
            for got, want in ((k[before[b]:], kx), (v[before[b]:], vx)):
                top = want.abs().amax(-1, keepdim=True)
                room = HALF * want.abs() + 2.0 ** -18 * top
                if self.fp8:
                    room = room * 1.1 + 2.0 ** -4 * want.abs() + 2.0 ** -9 * top / 224
                assert ((got - want).abs() <= room).all()
            for h in range(s.kv_heads):
                for i, p in enumerate(pages):
                    want, scale = ref.box(k[i * 64:(i + 1) * 64, h])
                    assert torch.equal(bounds[p, h], want) and float(unit[p, h]) == scale
            for i in range(n):
                length = before[b] + i + 1
                for h in range(s.kv_heads):
                    hs = slice(h * group, (h + 1) * group)
                    pages_now = table[b, :ref.pages_of(length)].long()
                    want = ref.select(q[row + i, hs].cpu(), bounds[pages_now, h], unit[pages_now, h], blocks.shape[2], 1, 1)
                    assert blocks[row + i, h].tolist() == want + [-1] * (blocks.shape[2] - len(want))
                    seen = torch.cat([torch.arange(p * 64, min(p * 64 + 64, length)) for p in want])
                    o, _, bound, _ = ref.attention_row(q[row + i, hs].double().cpu(), k[seen, h:h + 1], v[seen, h:h + 1],
                                                       s.scale, "fp8" if self.fp8 else "bf16", torch.bfloat16)
                    assert ((out[row + i, hs] - o).abs() <= bound).all()
            row += n


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (6, 3, 64)])
def test_prompts_steps_and_replay(fp8, heads, kv_heads, dim):
    s = layer_of(4, 1000, heads=heads, kv_heads=kv_heads, dim=dim, pages=3, fp8=fp8)
    shadow, before = Shadow(s, fp8), [0, 0, 0, 0]
    g = torch.Generator(device="cuda").manual_seed(3)
    kept, store = {}, s._store

    def noted(*a):
        kept["q"] = store(*a)
        return kept["q"]
    s._store = noted
    for counts in ([5, 0, 70, 64], [130, 1, 3, 0]):           # prompts, in two chunks
        x = torch.randn((sum(counts), heads + 2 * kv_heads, dim), generator=g, device="cuda").to(torch.bfloat16)
        out, blocks = s.prompt(x, counts)
        shadow.check(x, counts, kept["q"], out, blocks, before)
        before = [a + c for a, c in zip(before, counts)]
    s.step()
    shadow.check(s.qkv, [1] * 4, s.q, s.out, s.blocks, before)
    before = [a + 1 for a in before]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.step()
    for _ in range(3):                                        # the second and the last one take pages
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        shadow.check(s.qkv, [1] * 4, s.q, s.out, s.blocks, before)
        before = [a + 1 for a in before]
