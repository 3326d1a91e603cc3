"""One decode step of a sparse latent attention layer, with this library's calls in their order:

    norm + rotation of the indexer's queries and keys (with queries that are rotated only it would
    be a call for each), rotation of the attention's queries
    the new tokens' keys into the indexer's cache, their latents into the latent cache
    the indexer's logits and the k best positions of every request
    attention over those positions

Everything lives in buffers that the step keeps, so that it can be captured in a CUDA graph and
replayed with new inputs, lengths and tables.

    python examples/sparse_decode_step.py [--requests 64] [--context 32768] [--topk 2048]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_paged_gb300 as lib  # noqa: E402

INDEX_PAGE_BYTES = 8448          # 64 positions: 128 e4m3 codes each, then 64 fp32 scales


class SparseDecodeStep:
    """Caches, weights and buffers of one layer for `requests` decode requests of up to `context`
    positions.  The inputs of a step are the attributes `index_q` [B, 64, 128], `index_k`
    [B, 1, 128], `index_w` [B, 64], `latent` [B, 512], `rope` [B, 64], `q_latent` [B, H, 512],
    `q_rope` [B, H, 64], `positions` [B] (the new token's) and `block_table`; `run()` leaves the
    attention's latent output in `out` and its selection in `idx`."""

    def __init__(self, requests, context, heads=64, topk=2048, kv_dtype=lib.KV_FP8_E4M3, seed=0):
        B, dev = requests, "cuda"
        g = torch.Generator(device=dev).manual_seed(seed)
        self.B, self.W, self.heads, self.topk, self.kv = B, (context + 63) // 64, heads, topk, kv_dtype
        bf16 = dict(dtype=torch.bfloat16, device=dev)
        # the step's inputs
        x = torch.randn((B, 65, 128), generator=g, device=dev).to(torch.bfloat16)
        self.index_q, self.index_k = x[:, :64], x[:, 64:]
        self.index_w = torch.randn((B, 64), generator=g, device=dev) / 8
        c = torch.randn((B, 576), generator=g, device=dev).to(torch.bfloat16)
        self.latent, self.rope = c[:, :512], c[:, 512:]
        q = torch.randn((B, heads, 576), generator=g, device=dev).to(torch.bfloat16)
        self.q_latent, self.q_rope = q[..., :512], q[..., 512:]
        self.positions = torch.zeros(B, dtype=torch.int32, device=dev)
        # weights and the rotations' tables
        self.index_norm = [1 + 0.1 * torch.randn(128, generator=g, device=dev) for _ in range(2)]
        self.index_bias = [0.1 * torch.randn(128, generator=g, device=dev) for _ in range(2)]
        self.latent_norm = 1 + 0.1 * torch.randn(512, generator=g, device=dev)
        self.table = lib.rope_table(self.W * 64, 64)
        self.scale = 192 ** -0.5
        # caches: one pool of pages each, the same block table for both
        pages = B * self.W
        self.block_table = torch.randperm(pages, generator=g, device=dev).to(torch.int32).view(B, self.W)
        self.index_cache = torch.zeros((pages, INDEX_PAGE_BYTES), dtype=torch.uint8, device=dev)
        self.latent_cache = torch.zeros((pages, lib.LATENT_PAGE_BYTES[kv_dtype]), dtype=torch.uint8, device=dev)
        # what the step computes on the way
        self.index_q_out, self.index_k_out = torch.empty((B, 64, 128), **bf16), torch.empty((B, 1, 128), **bf16)
        self.q_rope_out = torch.empty((B, heads, 64), **bf16)
        self.seqlens = torch.zeros(B, dtype=torch.int32, device=dev)
        self.slots = torch.zeros(B, dtype=torch.int32, device=dev)
        self.idx = torch.empty((B, topk), dtype=torch.int32, device=dev)
        self.logits = torch.empty(B * self.W * 64, device=dev)
        self.out = torch.empty((B, heads, 512), **bf16)
        self.lse = torch.empty((B, heads), device=dev)
        self.workspace = torch.empty(lib.dsa_latent_attention_workspace(), device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self):
        B = self.B
        # the new token's slot and the length that includes it
        torch.add(self.positions, 1, out=self.seqlens)
        page = self.block_table.gather(1, (self.positions // 64).long()[:, None])[:, 0]
        torch.add(page * 64, self.positions % 64, out=self.slots)
        lib.qk_norm_rope(self.index_q, self.index_k, self.positions, self.table, norm=lib.NORM_LAYER,
                         q_weight=self.index_norm[0], k_weight=self.index_norm[1],
                         q_bias=self.index_bias[0], k_bias=self.index_bias[1],
                         q_out=self.index_q_out, k_out=self.index_k_out, dev_status=self.status)
        lib.qk_norm_rope(self.q_rope, None, self.positions, self.table, norm=lib.NORM_NONE,
                         interleaved=True, q_out=self.q_rope_out, dev_status=self.status)
        st = lib.dsa_kcache_store(self.index_k_out, self.slots, B, self.index_cache, INDEX_PAGE_BYTES,
                                  self.index_cache.shape[0], lib.KV_FP8_E4M3, 128, 64, self.status)
        if st != 0:
            raise lib.DsaError(st)
        lib.latent_store(self.latent, self.rope, self.slots, self.latent_cache, self.kv,
                         norm_weight=self.latent_norm, positions=self.positions, rope_table=self.table,
                         interleaved=True, dev_status=self.status)
        st = lib.dsa_indexer_topk_decode(
            self.index_q_out, self.index_w, self.index_cache, self.index_cache.data_ptr() + 8192,
            INDEX_PAGE_BYTES, self.index_cache.shape[0], lib.KV_FP8_E4M3, self.block_table, self.W,
            self.seqlens, B, 64, 128, 64, self.W, self.topk, self.idx, None, self.topk, self.logits,
            self.logits.numel(), self.status)
        if st != 0:
            raise lib.DsaError(st)
        return lib.latent_attention(self.q_latent, self.q_rope_out, self.latent_cache, self.kv,
                                    self.block_table, self.seqlens, self.scale, idx=self.idx, out=self.out,
                                    lse=self.lse, workspace=self.workspace, dev_status=self.status)


def fill(step, lengths, seed=1):
    """Write `lengths[b]` random tokens of each request into both caches."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, n in enumerate(lengths):
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        slots = (step.block_table[b].gather(0, (pos // 64).long()) * 64 + pos % 64).contiguous()
        k = torch.randn((n, 128), generator=g, device="cuda").to(torch.bfloat16)
        c = torch.randn((n, 576), generator=g, device="cuda").to(torch.bfloat16)
        st = lib.dsa_kcache_store(k, slots, n, step.index_cache, INDEX_PAGE_BYTES, step.index_cache.shape[0],
                                  lib.KV_FP8_E4M3, 128, 64, step.status)
        if st != 0:
            raise lib.DsaError(st)
        lib.latent_store(c[:, :512], c[:, 512:], slots, step.latent_cache, step.kv,
                         norm_weight=step.latent_norm, positions=pos, rope_table=step.table,
                         interleaved=True, dev_status=step.status)
        step.positions[b] = n


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--requests", type=int, default=64)
    ap.add_argument("--context", type=int, default=32768)
    ap.add_argument("--topk", type=int, default=2048)
    ap.add_argument("--kv", choices=["fp8", "bf16"], default="fp8")
    a = ap.parse_args()
    kv = lib.KV_FP8_E4M3 if a.kv == "fp8" else lib.KV_BF16
    step = SparseDecodeStep(a.requests, a.context, topk=a.topk, kv_dtype=kv)
    fill(step, [max(1, a.context * (b + 1) // a.requests - 1) for b in range(a.requests)])
    step.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    times = []
    for _ in range(20):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        times.append(begin.elapsed_time(end) * 1e3)
    if int(step.status):
        raise lib.DsaError(int(step.status))
    print(f"{a.requests} requests, context up to {a.context}, {a.topk} selected, {a.kv} cache: "
          f"{sorted(times)[len(times) // 2]:.1f} us a step")


if __name__ == "__main__":
    main()
