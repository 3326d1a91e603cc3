"""A layer of block-sparse attention with grouped heads over a paged cache of keys and values, with
this library's calls in their order:

    pages and slots of the new tokens from the requests' lengths
    norm + rotation of queries and keys
    the new tokens into the cache, the boxes around the keys of the pages that they touched
    the pages of every row and key head that may hold the largest scores
    attention over those pages

The same calls take a decode step (a token for every request) and a prompt's chunk (many; every
token is a row with its own causal length).  Everything of a decode step lives in buffers that the
layer keeps, so that it can be captured in a CUDA graph and replayed.

    python examples/block_sparse_step.py [--requests 64] [--context 32768] [--pages 32]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_paged_gb300 as lib  # noqa: E402


class BlockSparseLayer:
    """Cache, weights and buffers for `requests` requests of up to `context` tokens.  `qkv` [B, Hq + 2
    Hkv, D] is a decode step's input; `step()` leaves the attention's output in `out` and the
    selected pages in `blocks`, and the tokens count in `lengths` from then on."""

    def __init__(self, requests, context, heads=32, kv_heads=8, dim=128, pages=32, fp8=True, seed=0):
        B, H, dev = requests, kv_heads, "cuda"
        g = torch.Generator(device=dev).manual_seed(seed)
        self.B, self.W, self.heads, self.kv_heads, self.dim = B, (context + 63) // 64, heads, H, dim
        int32, bf16 = dict(dtype=torch.int32, device=dev), dict(dtype=torch.bfloat16, device=dev)
        count = B * self.W
        # the cache, head-major pages, and a box per page and key head
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        self.k_pool = torch.zeros((count, H, 64, dim), device=dev, dtype=torch.bfloat16).to(kind)
        self.v_pool = self.k_pool.clone()
        self.k_cache, self.v_cache = self.k_pool.transpose(1, 2), self.v_pool.transpose(1, 2)
        self.k_scale = torch.zeros((count, H, 64), device=dev) if fp8 else None
        self.v_scale = torch.zeros((count, H, 64), device=dev) if fp8 else None
        self.bounds = torch.zeros((count, H, 2, dim), dtype=torch.int8, device=dev)
        self.bound_scale = torch.zeros((count, H), device=dev)
        # requests: tokens held, their pages, and the pages that nobody has (the list's first `left`)
        self.lengths = torch.zeros(B, **int32)
        self.block_table = torch.full((B, self.W), -1, **int32)
        self.free = torch.randperm(count, generator=g, device=dev).to(torch.int32)
        self.places = torch.arange(count, device=dev)
        # weights
        self.q_norm = 1 + 0.1 * torch.randn(dim, generator=g, device=dev)
        self.k_norm = 1 + 0.1 * torch.randn(dim, generator=g, device=dev)
        self.table = lib.rope_table(self.W * 64, dim)
        self.scale = dim ** -0.5
        # a decode step's input and buffers
        self.qkv = torch.randn((B, heads + 2 * H, dim), generator=g, device=dev).to(torch.bfloat16)
        self.one = torch.ones(B, **int32)
        self.slots, self.positions = torch.zeros(B, **int32), torch.zeros(B, **int32)
        self.seqlens, self.cu, self.used = torch.zeros(B, **int32), torch.zeros(B + 1, **int32), torch.zeros(1, **int32)
        self.q, self.k = torch.empty((B, heads, dim), **bf16), torch.empty((B, H, dim), **bf16)
        self.blocks = torch.empty((B, H, pages), **int32)
        self.out, self.lse = torch.empty((B, heads, dim), **bf16), torch.empty((B, heads), device=dev)
        self.workspace = torch.empty(lib.dsa_paged_attention_workspace(heads, H, dim), device=dev)
        self.status = torch.zeros(1, **int32)

    def _take(self):
        """The pages that the last call gave out leave the free list's front."""
        at = (self.places + self.used).clamp(max=self.places.numel() - 1)
        self.free.copy_(self.free[at])

    def _store(self, qkv, positions, slots, seqlens, most, q=None, k=None):
        split = [self.heads, self.kv_heads, self.kv_heads]
        q_in, k_in, v = qkv.split(split, dim=1)
        q, k = lib.qk_norm_rope(q_in, k_in, positions, self.table, q_weight=self.q_norm, k_weight=self.k_norm,
                                q_out=q, k_out=k, dev_status=self.status)
        lib.kv_store(k, v, slots, self.k_cache, self.v_cache, k_scale=self.k_scale, v_scale=self.v_scale,
                     dev_status=self.status)
        lib.block_bounds(self.k_cache, self.block_table, self.lengths, seqlens, most, self.bounds, self.bound_scale,
                         k_scale=self.k_scale, dev_status=self.status)
        return q

    def _attend(self, q, table, seqlens, blocks, out=None, lse=None):
        lib.block_select(q, self.bounds, self.bound_scale, table, seqlens, blocks.shape[2], out=blocks,
                         dev_status=self.status)
        return lib.paged_attention(q, self.k_cache, self.v_cache, table, seqlens, self.scale, blocks=blocks,
                                   k_scale=self.k_scale, v_scale=self.v_scale, out=out, lse=lse,
                                   workspace=self.workspace, dev_status=self.status)

    def step(self):
        """One token for every request."""
        lib.request_slots(self.lengths, self.one, self.free, self.block_table, self.B, slots=self.slots,
                          positions=self.positions, seqlens=self.seqlens, cu_rows=self.cu, used=self.used,
                          dev_status=self.status)
        self._take()
        q = self._store(self.qkv, self.positions, self.slots, self.seqlens, 1, self.q, self.k)
        self._attend(q, self.block_table, self.seqlens, self.blocks, self.out, self.lse)
        self.lengths.copy_(self.seqlens)
        return self.out

    def prompt(self, qkv, counts):
        """counts[b] tokens of each request, requests in order; returns their attention and pages."""
        new = torch.tensor(counts, dtype=torch.int32, device="cuda")
        n = sum(counts)
        slots, positions, seqlens, _, _ = lib.request_slots(self.lengths, new, self.free, self.block_table, n,
                                                            used=self.used, dev_status=self.status)
        self._take()
        q = self._store(qkv, positions, slots, seqlens, max(counts))
        rows = torch.repeat_interleave(torch.arange(self.B, device="cuda"), new.long(), output_size=n)
        blocks = torch.empty((n, self.kv_heads, self.blocks.shape[2]), dtype=torch.int32, device="cuda")
        # every token reads up to itself
        out = self._attend(q, self.block_table[rows], positions + 1, blocks)
        self.lengths.copy_(seqlens)
        return out, blocks


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--context", type=int, default=32768)
    ap.add_argument("--pages", type=int, default=32)
    ap.add_argument("--kv", choices=["fp8", "bf16"], default="fp8")
    a = ap.parse_args()
    layer = BlockSparseLayer(a.requests, a.context, pages=a.pages, fp8=a.kv == "fp8")
    g = torch.Generator(device="cuda").manual_seed(1)
    width = layer.heads + 2 * layer.kv_heads
    lengths = [max(1, (a.context - 64) * (b + 1) // a.requests) for b in range(a.requests)]
    done = [0] * a.requests
    while done != lengths:                                # prompts in chunks of up to 4,096 tokens
        room, counts = 4096, []
        for have, want in zip(done, lengths):
            counts.append(min(room, want - have))
            room -= counts[-1]
        x = torch.randn((sum(counts), width, layer.dim), generator=g, device="cuda").to(torch.bfloat16)
        layer.prompt(x, counts)
        done = [d + c for d, c in zip(done, counts)]
    layer.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step()
    times = []
    for _ in range(20):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end) * 1e3)
    if int(layer.status):
        raise lib.DsaError(int(layer.status))
    print(f"{a.requests} requests, context up to {a.context}, {a.pages} pages of 64 selected, {a.kv} cache: "
          f"{sorted(times)[len(times) // 2]:.1f} us a step")


if __name__ == "__main__":
    main()
