"""GB300 (sm_103a) DSA indexer paged MQA-logits.

Thin Python binding of libdsa_indexer.so (``include/dsa_indexer.h``).  The
functions below carry the C names and only marshal arguments: tensors become
device pointers, the stream defaults to torch's current stream.  Every step
of the computation runs in the library's CUDA kernels; there is no CPU or
PyTorch fallback, and a missing library raises.

For each row r and position t < W*64:
``out[r, t] = scale(t) * sum_h w[r, h] * relu(q[r, h, :] . k(t))`` if
``t < seqlens[r]``, else ``-inf``.
"""
from __future__ import annotations

import ctypes

from . import _native

KV_FP8_E4M3 = 0
KV_BF16 = 1
H = 64
D = 128
PAGE = 64

STATUS = {
    0: "DSA_OK", 1: "DSA_ERR_INVALID_ARG", 2: "DSA_ERR_UNSUPPORTED",
    3: "DSA_ERR_MISALIGNED", 4: "DSA_ERR_CUDA", 5: "DSA_ERR_TIMEOUT",
    6: "DSA_ERR_BAD_PAGE", 7: "DSA_ERR_BAD_SEQLEN", 8: "DSA_ERR_BAD_POSITION",
}


class DsaError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(dsa_status_string(status))


def _p(x) -> int | None:
    """Device address of a tensor, or an int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor (the library takes device pointers)")
    return x.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class _AllocateOn:
    """Allocations for a call on `stream` (None: torch's current one; 0: the default stream).

    Within, torch allocates on that stream: the allocator then takes no memory that other streams
    may still be using, and once the call has dropped its own it goes to later work of that stream
    only.  ``returned`` marks an output, which leaves for a program on the current stream.
    """

    def __init__(self, stream, like):
        self.scope = self.current = None
        if stream is not None and like.is_cuda:
            import torch
            if isinstance(stream, int):
                stream = (torch.cuda.ExternalStream(stream, device=like.device) if stream
                          else torch.cuda.default_stream(like.device))
            self.current = torch.cuda.current_stream(like.device)
            self.scope = torch.cuda.stream(stream)

    def __enter__(self):
        if self.scope is not None:
            self.scope.__enter__()
        return self

    def __exit__(self, *error):
        if self.scope is not None:
            self.scope.__exit__(*error)

    def returned(self, x):
        if self.current is not None:
            x.record_stream(self.current)
        return x


def dsa_status_string(status: int) -> str:
    return _native.load().dsa_status_string(int(status)).decode()


def dsa_indexer_abi_version() -> int:
    return int(_native.load().dsa_indexer_abi_version())


def dsa_indexer_logits_decode(q, w, kcache, kscale, page_stride_bytes, num_pages,
                              kv_dtype, block_table, bt_stride, seqlens, B, H, D,
                              page_size, W, out, out_stride, dev_status=None,
                              stream=None) -> int:
    """C ``dsa_indexer_logits_decode``; returns its status code."""
    return int(_native.load().dsa_indexer_logits_decode(
        _p(q), _p(w), _p(kcache), _p(kscale), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), _p(block_table), int(bt_stride), _p(seqlens), int(B), int(H),
        int(D), int(page_size), int(W), _p(out), int(out_stride), _p(dev_status),
        _stream(stream)))


def dsa_indexer_logits_prefill(q, w, kcache, kscale, page_stride_bytes, num_pages,
                               kv_dtype, block_table, bt_stride, seqlens, n_q, H, D,
                               page_size, W, out, out_stride, dev_status=None,
                               stream=None) -> int:
    """C ``dsa_indexer_logits_prefill``; returns its status code."""
    return int(_native.load().dsa_indexer_logits_prefill(
        _p(q), _p(w), _p(kcache), _p(kscale), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), _p(block_table), int(bt_stride), _p(seqlens), int(n_q), int(H),
        int(D), int(page_size), int(W), _p(out), int(out_stride), _p(dev_status),
        _stream(stream)))


def dsa_indexer_logits_prefill_varlen(q, w, kcache, kscale, page_stride_bytes, num_pages,
                                      kv_dtype, block_table, bt_stride, cu_q, seqlens, H, D,
                                      page_size, W, out, out_stride, dev_status=None,
                                      stream=None) -> int:
    """C ``dsa_indexer_logits_prefill_varlen``; returns its status code.  `cu_q`
    is host data (a sequence of n_req + 1 ints); n_req = len(cu_q) - 1."""
    offs = [int(v) for v in cu_q]
    n_req = max(len(offs) - 1, 0)
    arr = (ctypes.c_int * max(len(offs), 1))(*offs)
    return int(_native.load().dsa_indexer_logits_prefill_varlen(
        _p(q), _p(w), _p(kcache), _p(kscale), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), _p(block_table), int(bt_stride),
        ctypes.cast(arr, ctypes.c_void_p).value if offs else None, n_req, _p(seqlens),
        int(H), int(D), int(page_size), int(W), _p(out), int(out_stride), _p(dev_status),
        _stream(stream)))


def dsa_indexer_topk_decode(q, w, kcache, kscale, page_stride_bytes, num_pages, kv_dtype,
                            block_table, bt_stride, seqlens, B, H, D, page_size, W, k_top,
                            topk_idx, topk_val, topk_stride, workspace, workspace_floats,
                            dev_status=None, stream=None) -> int:
    """C ``dsa_indexer_topk_decode``; returns its status code."""
    return int(_native.load().dsa_indexer_topk_decode(
        _p(q), _p(w), _p(kcache), _p(kscale), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), _p(block_table), int(bt_stride), _p(seqlens), int(B), int(H), int(D),
        int(page_size), int(W), int(k_top), _p(topk_idx), _p(topk_val), int(topk_stride),
        _p(workspace), int(workspace_floats), _p(dev_status), _stream(stream)))


TOPK_AUTO = 0
TOPK_TWO_PASS = 1
TOPK_FUSED = 2


def dsa_indexer_topk_decode_form(q, w, kcache, kscale, page_stride_bytes, num_pages, kv_dtype,
                                 block_table, bt_stride, seqlens, B, H, D, page_size, W, k_top,
                                 topk_idx, topk_val, topk_stride, workspace, workspace_floats,
                                 dev_status=None, form=TOPK_AUTO, stream=None) -> int:
    """C ``dsa_indexer_topk_decode_form``; returns its status code."""
    return int(_native.load().dsa_indexer_topk_decode_form(
        _p(q), _p(w), _p(kcache), _p(kscale), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), _p(block_table), int(bt_stride), _p(seqlens), int(B), int(H), int(D),
        int(page_size), int(W), int(k_top), _p(topk_idx), _p(topk_val), int(topk_stride),
        _p(workspace), int(workspace_floats), _p(dev_status), int(form), _stream(stream)))


def dsa_indexer_topk_decode_static(q, w, kcache, kscale, page_stride_bytes, num_pages,
                                   kv_dtype, block_table, bt_stride, seqlens, B, H, D,
                                   page_size, W, k_top, topk_idx, topk_val, topk_stride,
                                   dev_status=None, stream=None) -> int:
    """C ``dsa_indexer_topk_decode_static``; returns its status code."""
    return int(_native.load().dsa_indexer_topk_decode_static(
        _p(q), _p(w), _p(kcache), _p(kscale), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), _p(block_table), int(bt_stride), _p(seqlens), int(B), int(H), int(D),
        int(page_size), int(W), int(k_top), _p(topk_idx), _p(topk_val), int(topk_stride),
        _p(dev_status), _stream(stream)))


def dsa_kcache_store(k, slot_mapping, n, kcache, page_stride_bytes, num_pages, kv_dtype,
                     D, page_size, dev_status=None, stream=None) -> int:
    """C ``dsa_kcache_store``; returns its status code."""
    return int(_native.load().dsa_kcache_store(
        _p(k), _p(slot_mapping), int(n), _p(kcache), int(page_stride_bytes), int(num_pages),
        int(kv_dtype), int(D), int(page_size), _p(dev_status), _stream(stream)))


def indexer_logits(kind: str, q, w, kcache, kscale, page_stride_bytes, num_pages,
                   kv_dtype, block_table, bt_stride, seqlens, W, out=None,
                   dev_status=None, stream=None):
    """Allocate the [rows, W*64] fp32 output (if not given) and run one call.

    ``kind`` is "decode" or "prefill".  Raises DsaError on a host-side error.
    """
    import torch
    rows = int(seqlens.shape[0])
    if out is None:
        with _AllocateOn(stream, seqlens) as on:
            out = on.returned(seqlens.new_empty((rows, W * PAGE), dtype=torch.float32))
    fn = dsa_indexer_logits_decode if kind == "decode" else dsa_indexer_logits_prefill
    st = fn(q, w, kcache, kscale, page_stride_bytes, num_pages, kv_dtype, block_table,
            bt_stride, seqlens, rows, H, D, PAGE, W, out, out.stride(0), dev_status, stream)
    if st != 0:
        raise DsaError(st)
    return out


# ---- around the sparse attention: norm + rotation, latent cache, attention ----

BF16 = 0
FP16 = 1
FP32 = 2
NORM_NONE = 0
NORM_RMS = 1
NORM_LAYER = 2
LATENT = 512
ROPE = 64
LATENT_PAGE_BYTES = {KV_FP8_E4M3: 41984, KV_BF16: 73728}


def dsa_qk_norm_rope(q, q_token_stride, q_head_stride, Hq, k, k_token_stride, k_head_stride, Hk,
                     T, D, dtype, norm, q_weight, k_weight, q_bias, k_bias, eps, positions,
                     rope_table, max_pos, rot_dims, rot_offset, interleaved, q_out,
                     qo_token_stride, qo_head_stride, k_out, ko_token_stride, ko_head_stride,
                     dev_status=None, stream=None) -> int:
    """C ``dsa_qk_norm_rope``; returns its status code."""
    return _native.load().dsa_qk_norm_rope(
        _p(q), q_token_stride, q_head_stride, Hq, _p(k), k_token_stride, k_head_stride, Hk, T, D,
        dtype, norm, _p(q_weight), _p(k_weight), _p(q_bias), _p(k_bias), eps, _p(positions),
        _p(rope_table), max_pos, rot_dims, rot_offset, int(interleaved), _p(q_out),
        qo_token_stride, qo_head_stride, _p(k_out), ko_token_stride, ko_head_stride,
        _p(dev_status), _stream(stream))


def dsa_latent_store(latent, latent_stride, rope, rope_stride, n, latent_dim, rope_dim,
                     norm_weight, eps, positions, rope_table, max_pos, interleaved, slot_mapping,
                     cache, page_stride_bytes, num_pages, kv_dtype, page_size, dev_status=None,
                     stream=None) -> int:
    """C ``dsa_latent_store``; returns its status code."""
    return _native.load().dsa_latent_store(
        _p(latent), latent_stride, _p(rope), rope_stride, n, latent_dim, rope_dim,
        _p(norm_weight), eps, _p(positions), _p(rope_table), max_pos, int(interleaved),
        _p(slot_mapping), _p(cache), page_stride_bytes, num_pages, kv_dtype, page_size,
        _p(dev_status), _stream(stream))


def dsa_latent_load(cache, page_stride_bytes, num_pages, kv_dtype, page_size, block_table,
                    bt_stride, W, starts, cu_rows, n_req, n, latent_dim, rope_dim, out,
                    out_stride, dev_status=None, stream=None) -> int:
    """C ``dsa_latent_load``; returns its status code."""
    return _native.load().dsa_latent_load(
        _p(cache), page_stride_bytes, num_pages, kv_dtype, page_size, _p(block_table), bt_stride,
        W, _p(starts), _p(cu_rows), n_req, n, latent_dim, rope_dim, _p(out), out_stride,
        _p(dev_status), _stream(stream))


def dsa_latent_attention(q_latent, ql_row_stride, ql_head_stride, q_rope, qr_row_stride,
                         qr_head_stride, rows, H, latent_dim, rope_dim, scale, cache,
                         page_stride_bytes, num_pages, kv_dtype, page_size, block_table,
                         bt_stride, W, seqlens, idx, idx_stride, k, out, out_row_stride,
                         out_head_stride, lse, workspace, workspace_floats, dev_status=None,
                         stream=None) -> int:
    """C ``dsa_latent_attention``; returns its status code."""
    return _native.load().dsa_latent_attention(
        _p(q_latent), ql_row_stride, ql_head_stride, _p(q_rope), qr_row_stride, qr_head_stride,
        rows, H, latent_dim, rope_dim, scale, _p(cache), page_stride_bytes, num_pages, kv_dtype,
        page_size, _p(block_table), bt_stride, W, _p(seqlens), _p(idx), idx_stride, k, _p(out),
        out_row_stride, out_head_stride, _p(lse), _p(workspace), workspace_floats,
        _p(dev_status), _stream(stream))


def dsa_latent_attention_workspace() -> int:
    """C ``dsa_latent_attention_workspace``: floats for the current device, -1 without one."""
    return int(_native.load().dsa_latent_attention_workspace())


_calls = None


def _tensor_calls():
    global _calls
    if _calls is None:
        _calls = _native.load_calls()
    return _calls


# The tensor-level calls run on torch's current stream unless `stream` names another (a
# torch.cuda.Stream, or a cudaStream_t as an int).  What they allocate belongs to that stream; the
# order between it and the streams of the tensors that are given, and those tensors' lives, are
# the caller's to keep.

def _stream_address(stream):
    return stream if stream is None or isinstance(stream, int) else stream.cuda_stream


def rope_table(max_pos, rot_dims, base=10000.0, device="cuda"):
    """The fp32 [max_pos, rot_dims] table of the rotations: per position rot_dims/2 cosines, then
    the sines, of position * base^(-2i/rot_dims); the angles are taken in 64 bits."""
    import torch
    freq = float(base) ** (-torch.arange(0, rot_dims, 2, dtype=torch.float64, device=device) / rot_dims)
    angle = torch.arange(max_pos, dtype=torch.float64, device=device)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def qk_norm_rope(q, k, positions=None, table=None, *, rot_dims=None, rot_offset=0,
                 interleaved=False, norm=NORM_RMS, q_weight=None, k_weight=None, q_bias=None,
                 k_bias=None, eps=1e-6, q_out=None, k_out=None, dev_status=None, stream=None):
    """Norm and rotate queries [T, Hq, D] and keys [T, Hk, D] per head, in one kernel.

    The last dimension is contiguous, the others may be strided; ``k`` may be None.  One ``norm``
    for both: with different ones, a call for each.  ``table`` as ``rope_table`` makes it.
    Outputs are allocated unless given (in place: pass q and k).  Returns (q_out, k_out).  Raises
    DsaError on a host-side error.
    """
    if rot_dims is not None and table is not None and rot_dims != table.shape[1]:
        raise ValueError("rot_dims: the table's width")
    if q_out is None or (k_out is None and k is not None):
        with _AllocateOn(stream, q) as on:
            if q_out is None:
                q_out = on.returned(q.new_empty(q.shape))
            if k_out is None and k is not None:
                k_out = on.returned(k.new_empty(k.shape))
    status = (_calls or _tensor_calls()).qk_norm_rope(
        q, k, positions, table, rot_offset, interleaved, norm, q_weight, k_weight, q_bias, k_bias,
        eps, q_out, k_out, dev_status, _stream_address(stream))
    if status:
        raise DsaError(status)
    return q_out, k_out


def latent_store(latent, rope, slot_mapping, cache, kv_dtype, *, norm_weight=None, eps=1e-6,
                 positions=None, rope_table=None, interleaved=False, dev_status=None, stream=None):
    """Write n tokens (latent [n, 512], rope [n, 64], bf16) into their slots of ``cache``.

    Optionally normalises the latent and rotates the other part on the way.  ``cache``: uint8
    [pages, LATENT_PAGE_BYTES[kv_dtype]].  Raises DsaError on a host-side error.
    """
    status = (_calls or _tensor_calls()).latent_store(
        latent, rope, slot_mapping, cache, kv_dtype, norm_weight, eps, positions, rope_table,
        interleaved, dev_status, _stream_address(stream))
    if status:
        raise DsaError(status)
    return cache


def latent_load(cache, kv_dtype, block_table, cu_rows, n, *, starts=None, out=None,
                dev_status=None, stream=None):
    """Read ranges of cached tokens back as bf16 [n, 576] (latent, then rotated part).

    ``cu_rows`` int32 [requests + 1] on the device: request r's rows of the output.  Raises
    DsaError on a host-side error.
    """
    if out is None:
        import torch
        with _AllocateOn(stream, cache) as on:
            out = on.returned(cache.new_empty((n, LATENT + ROPE), dtype=torch.bfloat16))
    status = (_calls or _tensor_calls()).latent_load(
        cache, kv_dtype, block_table, cu_rows, n, starts, out, dev_status, _stream_address(stream))
    if status:
        raise DsaError(status)
    return out


def latent_attention(q_latent, q_rope, cache, kv_dtype, block_table, seqlens, scale, *, idx=None,
                     out=None, lse=None, workspace=None, dev_status=None, stream=None):
    """Attention of [rows, H] query heads over the latent cache, in the absorbed form.

    Over every position below ``seqlens``, or over the selection lists ``idx`` (int32 [rows, k],
    k >= 1, as the top-k calls write them; a row whose entries are all -1 gives zeros and lse
    -inf).  Returns out, bf16 [rows, H, 512]; ``lse`` (fp32 [rows, H])
    is written when given.  ``block_table`` has a row per query row, or one for all; a prompt's
    tokens of one of several requests repeat its row.  Raises DsaError on a host-side error.
    """
    if out is None or workspace is None:
        import torch
        with _AllocateOn(stream, q_latent) as on:
            if out is None:
                out = on.returned(q_latent.new_empty(q_latent.shape))
            if workspace is None:
                workspace = q_latent.new_empty(max(dsa_latent_attention_workspace(), 0),
                                               dtype=torch.float32)
    status = (_calls or _tensor_calls()).latent_attention(
        q_latent, q_rope, cache, kv_dtype, block_table, seqlens, scale, idx, out, lse, workspace,
        dev_status, _stream_address(stream))
    if status:
        raise DsaError(status)
    return out
