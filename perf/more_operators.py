"""Performance cases of attention over a paged cache of keys and values, and of what serves it.

Four operators of a serving step with grouped heads (Hq query heads share Hkv
key and value heads), each reached through ``sparse_attention_paged_gb300``:

``request_slots``
    From the requests' cached and new lengths: pages for the new tokens out of
    a free list into the block table, and every new token's slot and position.
``kv_cache``
    New tokens into their slots of the paged cache (``kv_store``; as they are,
    or e4m3 with a scale per token and head), then the box around the keys of
    every page that they touched (``block_bounds``).
``block_select``
    The k pages of every row and key head whose boxes allow the largest scores
    of the group's queries.
``paged_attention``
    Attention of one new token per row over its cached tokens: all of them, or
    those of the pages that a list names.

``own`` chooses between the plain form (elementary torch operations in 32
bits, rounded once at the end) and the library's calls.
"""
import math

import torch

own = False

PAGE = 64       # tokens per page
GRID = 20       # bits of the grid that a group's queries are summed on
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _slots(name, requests, low, high, context):
    """`requests` with up to `context` cached tokens, each with `low` to `high` new ones."""
    return {"name": name, "op": "request_slots", "requests": requests, "low": low, "high": high,
            "context": context}


def _cache(name, requests, tokens, context, kv_heads, dim, kv, dtype):
    return {"name": name, "op": "kv_cache", "requests": requests, "tokens": tokens, "context": context,
            "kv_heads": kv_heads, "dim": dim, "kv": kv, "dtype": dtype}


def _select(name, rows, heads, kv_heads, dim, k, min_len, max_len, prefill, dtype):
    return {"name": name, "op": "block_select", "rows": rows, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "k": k, "min_len": min_len, "max_len": max_len, "prefill": prefill, "dtype": dtype}


def _attention(name, rows, heads, kv_heads, dim, kv, k, min_len, max_len, prefill, dtype):
    return {"name": name, "op": "paged_attention", "rows": rows, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "kv": kv, "k": k, "min_len": min_len, "max_len": max_len, "prefill": prefill,
            "dtype": dtype}


def listed():
    return [
        # one decode step of 64 requests: a token each
        _slots("slots_decode_64", 64, 1, 1, 131072),
        # prompts of 23 requests, some of them after earlier chunks or a shared prefix
        _slots("slots_prompts_23", 23, 0, 1953, 8192),
        # one decode step of 64 short requests into an fp8 cache
        _cache("kv_fp8_decode_64", 64, 1, 65, 8, 128, "fp8", "bf16"),
        # a prefill of 22,528 tokens into a bf16 cache
        _cache("kv_bf16_prefill_22528", 1, 22528, 22528, 8, 128, "bf16", "bf16"),
        # decode of 64 long requests: 32 pages (2,048 tokens) of up to 2,048
        _select("select_decode_b64_w2048", 64, 64, 8, 128, 32, 4096, 131072, False, "bf16"),
        # a prefill chunk over a shared context, every query token with its own pages
        _select("select_prefill_1024", 1024, 32, 8, 128, 16, 0, 22528, True, "bf16"),
        # the smallest call: one short request, few heads of a split model
        _attention("attn_bf16_b1_1000", 1, 8, 2, 128, "bf16", 0, 1000, 1000, False, "bf16"),
        # decode over selected pages of long requests, fp8 cache
        _attention("attn_blocks_fp8_b64_k32", 64, 64, 8, 128, "fp8", 32, 4096, 32768, False, "bf16"),
        # decode over every token, lengths log-uniform
        _attention("attn_dense_bf16_b64", 64, 32, 8, 128, "bf16", 0, 512, 32768, False, "bf16"),
        # decode of one long request, fp8 cache
        _attention("attn_dense_fp8_b1_131072", 1, 64, 8, 128, "fp8", 0, 131072, 131072, False, "bf16"),
        # odd sizes: groups of 7 heads, smaller heads, lengths from one token
        _attention("attn_dense_fp16_b19", 19, 35, 5, 64, "fp16", 0, 1, 9001, False, "fp16"),
        # a prefill chunk over a shared context, every query token with its own pages
        _attention("attn_prefill_bf16_1024_k16", 1024, 32, 4, 128, "bf16", 16, 0, 22528, True, "bf16"),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["request_slots", "kv_cache", "block_select", "paged_attention", "paged_attention"])
    dim, dtype = rng.choice([64, 128]), rng.choice(["bf16", "fp16"])
    kv = rng.choice([dtype, "fp8"])
    kv_heads = rng.randint(1, 8)
    group = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    if kind == "request_slots":
        requests = _log_int(rng, 1, 512)
        high = rng.choice([1, _log_int(rng, 1, 22528 // requests)])
        case = _slots("", requests, rng.choice([0, high]), high, _log_int(rng, 1, 131072))
    elif kind == "kv_cache":
        requests = _log_int(rng, 1, 64)
        context = _log_int(rng, 1, 22528 // requests)
        case = _cache("", requests, _log_int(rng, 1, context), context, kv_heads, dim, kv, dtype)
    elif kind == "block_select":
        prefill = rng.random() < 0.5
        rows = _log_int(rng, 2, 1024) if prefill else _log_int(rng, 1, 64)
        top = rows + _log_int(rng, 1, 22528 - rows) if prefill else _log_int(rng, 64, 131072)
        case = _select("", rows, group * kv_heads, kv_heads, dim, _log_int(rng, 2, 64),
                       0 if prefill else max(1, top // 32), top, prefill, dtype)
    else:
        prefill = rng.random() < 0.25
        if prefill:
            rows = _log_int(rng, 2, 1024)
            top, k = rows + _log_int(rng, 1, 22528 - rows), _log_int(rng, 1, 16)
            kv_heads = min(kv_heads, 4)
        else:
            rows, k = _log_int(rng, 1, 64), rng.choice([0, _log_int(rng, 1, 64)])
            top = _log_int(rng, 1, 32768 if rows > 2 else 131072)
        case = _attention("", rows, group * kv_heads, kv_heads, dim, kv, k,
                          0 if prefill else max(1, top // 64), top, prefill, dtype)
    del case["name"]
    return case


def _spread(n, low, high):
    """n lengths from low to high, log-uniform (even quantiles); one alone has the highest."""
    if n == 1:
        return [high]
    ratio = math.log(high / low)
    return [min(high, int(low * math.exp(ratio * i / (n - 1)))) for i in range(n)]


def _lengths(case):
    """Lengths of the rows: the causal limits of a prefill, else log-uniform."""
    rows, low, high = case["rows"], case["min_len"], case["max_len"]
    return [high - rows + 1 + i for i in range(rows)] if case["prefill"] else _spread(rows, low, high)


def _new_and_cached(case):
    """New and cached tokens of each request of a request_slots case."""
    n, low, high = case["requests"], case["low"], case["high"]
    new = [low + (high - low) * ((7 * i + 3) % n + 1) // n for i in range(n)]
    return new, [(case["context"] * ((5 * i + 1) % (n + 1))) // (n + 1) for i in range(n)]


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _block_tables(lens, g):
    """(block table [B, W], pages in all) of requests whose pages lie anywhere in the pool."""
    used = [_pages(v) for v in lens]
    W, pages = max(1, max(used)), max(1, sum(used))
    perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(used, device="cuda")
    at = (n.cumsum(0) - n)[:, None] + torch.arange(W, device="cuda")
    filled = torch.arange(W, device="cuda") < n[:, None]
    return torch.where(filled, perm[at.clamp(max=pages - 1)], torch.zeros_like(perm[:1])).contiguous(), pages


def _scales(top):
    """The smallest power of two, 2^-126 at least, that brings `top` to at most 448."""
    mantissa, exponent = torch.frexp(top)                 # top = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp(-126, 127)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, -126))


def _pool(pages, heads, dim, kv, g):
    """A pool [pages, heads, 64, dim] of random tokens, and its scales [pages, heads, 64] (fp8)."""
    pool = torch.empty((pages, heads, PAGE, dim), dtype=TYPES[kv], device="cuda")
    scale = torch.empty((pages, heads, PAGE), device="cuda") if kv == "fp8" else None
    step = max(1, (1 << 27) // (heads * PAGE * dim))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        x = torch.randn((n, heads, PAGE, dim), generator=g, device="cuda")
        if kv == "fp8":
            s = _scales(x.abs().amax(-1))
            scale[at:at + n] = s
            x = x / s[..., None]
        pool[at:at + n] = x.to(TYPES[kv])
    return pool, scale


def _prepare_slots(case, g):
    new, cached = _new_and_cached(case)
    B, n = case["requests"], sum(new)
    W = max(1, max(_pages(a + b) for a, b in zip(new, cached)))
    held = sum(_pages(c) for c in cached)
    wanted = sum(_pages(a + b) - _pages(b) for a, b in zip(new, cached))
    perm = torch.randperm(held + wanted + 100, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor([_pages(c) for c in cached], device="cuda")
    at = (count.cumsum(0) - count)[:, None] + torch.arange(W, device="cuda")
    filled = torch.arange(W, device="cuda") < count[:, None]
    return {"lengths": _int32(cached), "new": _int32(new), "free": perm[held:].contiguous(),
            "table": torch.where(filled, perm[at.clamp(max=max(held - 1, 0))], -1).contiguous(),
            # the step's buffers hold some tokens more, as those of a captured step do
            "n": n + 7, "slots": torch.empty(n + 7, dtype=torch.int32, device="cuda"),
            "positions": torch.empty(n + 7, dtype=torch.int32, device="cuda"),
            "seqlens": torch.empty(B, dtype=torch.int32, device="cuda"),
            "cu": torch.empty(B + 1, dtype=torch.int32, device="cuda"),
            "used": torch.empty(1, dtype=torch.int32, device="cuda")}


def _prepare_cache(case, g):
    B, n, L, H, D = case["requests"], case["tokens"], case["context"], case["kv_heads"], case["dim"]
    table, pages = _block_tables([L] * B, g)
    pos = torch.arange(L - n, L, device="cuda").expand(B, n)   # the last n of each request are new
    slots = table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE
    k_pool, k_scale = _pool(pages, H, D, case["kv"], g)
    v_pool, v_scale = _pool(pages, H, D, case["kv"], g)
    # one projection's output, heads side by side: keys, then values
    size = torch.exp(0.5 * torch.randn((B * n, 2 * H, 1), generator=g, device="cuda"))
    x = (torch.randn((B * n, 2 * H, D), generator=g, device="cuda") * size).to(TYPES[case["dtype"]])
    return {"k": x[:, :H], "v": x[:, H:], "slots": slots.reshape(-1).to(torch.int32), "table": table,
            "k_pool": k_pool, "v_pool": v_pool, "k_scale": k_scale, "v_scale": v_scale,
            "starts": torch.full((B,), L - n, dtype=torch.int32, device="cuda"),
            "seqlens": torch.full((B,), L, dtype=torch.int32, device="cuda"),
            "bounds": torch.zeros((pages, H, 2, D), dtype=torch.int8, device="cuda"),
            "bound_scale": torch.zeros((pages, H), device="cuda")}


def _queries(case, g):
    """Queries [rows, heads, dim] as a slice of one projection's output."""
    R, H, D = case["rows"], case["heads"], case["dim"]
    x = torch.randn((R, H + 2 * case["kv_heads"], D), generator=g, device="cuda")
    return x.to(TYPES[case["dtype"]])[:, :H]


def _rows_table(case, g):
    """(lengths, block table, pages): a row per request, or one row that a prefill's tokens share."""
    lens = _lengths(case)
    table, pages = _block_tables([max(lens)] if case["prefill"] else lens, g)
    return lens, table, pages


def _prepare_select(case, g):
    lens, table, pages = _rows_table(case, g)
    H, D = case["kv_heads"], case["dim"]
    # boxes around 64 standard normal keys, in steps of 2^-5
    half = (2.4 + 0.4 * torch.randn((pages, H, 2, D), generator=g, device="cuda")).clamp(0, 3.9)
    bounds = torch.ceil(half * 32)
    bounds[:, :, 1] *= -1
    scale = torch.ldexp(torch.ones((pages, H), device="cuda"),
                        torch.randint(-6, -4, (pages, H), generator=g, device="cuda"))
    return {"q": _queries(case, g), "bounds": bounds.to(torch.int8), "bound_scale": scale, "table": table,
            "seqlens": _int32(lens),
            "out": torch.empty((case["rows"], H, case["k"]), dtype=torch.int32, device="cuda")}


def _prepare_attention(case, g):
    lens, table, pages = _rows_table(case, g)
    R, H, D, k = case["rows"], case["kv_heads"], case["dim"], case["k"]
    seqlens = _int32(lens)
    blocks = None
    if k:
        n, W = _pages(seqlens.long())[:, None, None], max(k, table.shape[1])
        keys = torch.rand((R, H, W), generator=g, device="cuda")
        index = torch.arange(W, device="cuda")
        keys = torch.where(index == n - 1, 2.0, keys)           # the newest page is always among them
        keys = torch.where(index < n, keys, -1.0)
        best, where = keys.topk(k, dim=-1)
        where = torch.where(best >= 0, where, W).sort(dim=-1).values
        blocks = torch.where(where < W, where, -1).to(torch.int32)
    k_pool, k_scale = _pool(pages, H, D, case["kv"], g)
    v_pool, v_scale = _pool(pages, H, D, case["kv"], g)
    q = _queries(case, g)
    state = {"q": q, "k_pool": k_pool, "v_pool": v_pool, "k_scale": k_scale, "v_scale": v_scale, "table": table,
             "seqlens": seqlens, "blocks": blocks, "scale": D ** -0.5,
             "out": torch.empty((R, case["heads"], D), dtype=q.dtype, device="cuda"),
             "lse": torch.empty((R, case["heads"]), device="cuda")}
    # partial results of two pieces of a head group per SM and CTA on it, with a record each
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    group = case["heads"] // H
    state["workspace"] = torch.empty(sms * 4 * 2 * (group * (D + 4) + 4), device="cuda")
    return state


PREPARE = {"request_slots": _prepare_slots, "kv_cache": _prepare_cache, "block_select": _prepare_select,
           "paged_attention": _prepare_attention}


def prepare(case, seed):
    return {"case": dict(case), **PREPARE[case["op"]](case, _generator(seed))}


# ---------------------------------------------------------------------------
# one pass, plain
# ---------------------------------------------------------------------------

def _plain_slots(s):
    cached, new, table, n = s["lengths"].long(), s["new"].long(), s["table"], s["n"]
    B, W = table.shape
    index = torch.arange(W, device=table.device)
    have, want = _pages(cached), _pages(cached + new)
    before = (want - have).cumsum(0) - (want - have)
    at = (before[:, None] + index - have[:, None]).clamp(0, s["free"].shape[0] - 1)
    fresh = (index >= have[:, None]) & (index < want[:, None])
    table.copy_(torch.where(fresh, s["free"][at], table))
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    i = torch.arange(n, device=table.device)
    row = torch.searchsorted(cu[1:], i, right=True).clamp(max=B - 1)
    live = i < cu[-1]
    pos = torch.where(live, cached[row] + i - cu[row], 0)
    slot = torch.where(live, table[row, pos // PAGE].long() * PAGE + pos % PAGE, -1)
    int32 = torch.int32
    return (table, slot.to(int32), pos.to(int32), (cached + new).to(int32), cu.to(int32),
            (want - have).sum().to(int32).view(1))


def _plain_store(x, slots, pool, scale):
    page, slot = slots.long() // PAGE, slots.long() % PAGE
    if scale is None:
        pool[page, :, slot] = x
        return
    v = x.float()
    s = _scales(v.abs().amax(-1))
    scale[page, :, slot] = s
    pool.view(torch.uint8)[page, :, slot] = (v / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _values(pool, scale, *at):
    """Values of pool[at] in 32 bits."""
    if scale is None:
        return pool[at].float()
    return pool.view(torch.uint8)[at].view(torch.float8_e4m3fn).float() * scale[at][..., None]


def _plain_cache(s):
    _plain_store(s["k"], s["slots"], s["k_pool"], s["k_scale"])
    _plain_store(s["v"], s["slots"], s["v_pool"], s["v_scale"])
    # the pages that hold new tokens: every request's from the first one on
    first = (s["case"]["context"] - s["case"]["tokens"]) // PAGE
    index = torch.arange(first, s["table"].shape[1], device="cuda")
    left = (s["seqlens"].long()[:, None] - index * PAGE).flatten()
    page = s["table"][:, first:].long().flatten()
    keys = _values(s["k_pool"], s["k_scale"], page)                               # [n, H, 64, D]
    seen = (torch.arange(PAGE, device="cuda") < left[:, None])[:, None, :, None]
    high = torch.where(seen, keys, -math.inf).amax(2)
    low = torch.where(seen, keys, math.inf).amin(2)
    top = torch.maximum(high.abs(), low.abs()).amax(-1)
    mantissa, exponent = torch.frexp(top)                                         # 127 * 2^e >= top
    e = torch.where(mantissa <= 127 / 128, exponent - 7, exponent - 6).clamp(min=-126)
    unit = torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, -126))
    s["bounds"][page, :, 0] = torch.ceil(high / unit[..., None]).to(torch.int8)
    s["bounds"][page, :, 1] = torch.floor(low / unit[..., None]).to(torch.int8)
    s["bound_scale"][page] = unit
    return _cache_outputs(s)


def _cache_outputs(s):
    found = [s["k_pool"], s["v_pool"], s["bounds"], s["bound_scale"]]
    return found + ([] if s["k_scale"] is None else [s["k_scale"], s["v_scale"]])


def _plain_select(s):
    case, k = s["case"], s["case"]["k"]
    R, H, D = case["rows"], case["kv_heads"], case["dim"]
    # the group's queries on a grid of 2^-20 of their largest, positive and negative parts summed
    q = s["q"].view(R, H, -1, D).double()
    _, exponent = torch.frexp(q.abs().amax((2, 3), keepdim=True))
    grid = torch.round(torch.ldexp(q, GRID - exponent))
    parts = torch.stack([grid.clamp(min=0).sum(2), (-grid).clamp(min=0).sum(2)], 2)     # [R, H, 2, D]
    top = parts.amax((2, 3), keepdim=True)
    shift = torch.ceil(torch.log2(top.clamp(min=127) / 127)).clamp(min=0)
    codes = torch.ceil(parts / torch.exp2(shift)).float()
    codes[:, :, 1] *= -1                                                          # [R, H, 2, D]
    table = s["table"].long()
    boxes = s["bounds"][table].float()                                            # [., W, H, 2, D]
    dot = torch.einsum("rhcd,whcd->rhw", codes, boxes[0]) if case["prefill"] else \
        torch.einsum("rhcd,rwhcd->rhw", codes, boxes)
    score = dot * s["bound_scale"][table].transpose(1, 2)
    W = max(k, table.shape[1])
    score = torch.nn.functional.pad(score, (0, W - table.shape[1]))
    n, index = _pages(s["seqlens"].long())[:, None, None], torch.arange(W, device="cuda")
    score = torch.where((index < 1) | (index == n - 1), math.inf, score)          # the first and the newest
    score = torch.where(index < n, score, -math.inf)
    best, order = score.sort(dim=-1, descending=True, stable=True)
    order = torch.where(best[..., :k] > -math.inf, order[..., :k], W).sort(dim=-1).values
    return torch.where(order < W, order, -1).to(torch.int32)


def _plain_attention(s):
    case = s["case"]
    R, H, D = case["rows"], case["kv_heads"], case["dim"]
    table, length = s["table"].long(), s["seqlens"].long()[:, None, None, None]
    if s["blocks"] is None:
        block = torch.arange(table.shape[1], device="cuda").expand(R, H, -1)
    else:
        block = s["blocks"].long()
    seen = (block >= 0)[..., None] & (block[..., None] * PAGE + torch.arange(PAGE, device="cuda") < length)
    page = table[:, None].expand(R, H, -1).gather(2, block.clamp(min=0))
    head = torch.arange(H, device="cuda")[:, None]
    seen = seen.flatten(2)                                                        # [R, H, T]
    q = s["q"].view(R, H, -1, D).float()
    keys = _values(s["k_pool"], s["k_scale"], page, head).flatten(2, 3)           # [R, H, T, D]
    score = (q @ keys.transpose(2, 3)) * s["scale"]
    del keys
    score = torch.where(seen[:, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    values = _values(s["v_pool"], s["v_scale"], page, head).flatten(2, 3)
    out = (p @ values) / torch.where(total > 0, total, 1.0)
    return out.view(R, -1, D).to(s["q"].dtype), (top + torch.log(total)).view(R, -1)


# ---------------------------------------------------------------------------
# one pass, the library's calls
# ---------------------------------------------------------------------------

def _own_slots(s):
    import sparse_attention_paged_gb300 as lib
    lib.request_slots(s["lengths"], s["new"], s["free"], s["table"], s["n"], slots=s["slots"],
                      positions=s["positions"], seqlens=s["seqlens"], cu_rows=s["cu"], used=s["used"])
    return s["table"], s["slots"], s["positions"], s["seqlens"], s["cu"], s["used"]


def _own_cache(s):
    import sparse_attention_paged_gb300 as lib
    k_cache, v_cache = s["k_pool"].transpose(1, 2), s["v_pool"].transpose(1, 2)
    lib.kv_store(s["k"], s["v"], s["slots"], k_cache, v_cache, k_scale=s["k_scale"], v_scale=s["v_scale"])
    lib.block_bounds(k_cache, s["table"], s["starts"], s["seqlens"], s["case"]["tokens"], s["bounds"],
                     s["bound_scale"], k_scale=s["k_scale"])
    return _cache_outputs(s)


def _own_select(s):
    import sparse_attention_paged_gb300 as lib
    return lib.block_select(s["q"], s["bounds"], s["bound_scale"], s["table"], s["seqlens"], s["case"]["k"],
                            first=1, last=1, out=s["out"])


def _own_attention(s):
    import sparse_attention_paged_gb300 as lib
    lib.paged_attention(s["q"], s["k_pool"].transpose(1, 2), s["v_pool"].transpose(1, 2), s["table"], s["seqlens"],
                        s["scale"], blocks=s["blocks"], k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"],
                        lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


PASSES = {"request_slots": (_plain_slots, _own_slots), "kv_cache": (_plain_cache, _own_cache),
          "block_select": (_plain_select, _own_select), "paged_attention": (_plain_attention, _own_attention)}


def run(state):
    return PASSES[state["case"]["op"]][1 if own else 0](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "request_slots":
        new, cached = _new_and_cached(case)
        fresh = sum(_pages(a + b) - _pages(b) for a, b in zip(new, cached))
        return {"bytes": 16 * case["requests"] + 8 * fresh + 8 * (sum(new) + 7), "flops": 4 * sum(new)}
    if case["op"] == "kv_cache":
        B, n, L, H, D = case["requests"], case["tokens"], case["context"], case["kv_heads"], case["dim"]
        token = D * BYTES[case["kv"]] + (4 if case["kv"] == "fp8" else 0)
        touched = _pages(L) - (L - n) // PAGE
        earlier = (L - n) % PAGE                      # keys that the first touched page held before
        return {"bytes": B * H * (2 * n * (2 * D + token) + earlier * token + touched * (2 * D + 4)) + 4 * B * n,
                "flops": B * H * D * (2 * n + 2 * (n + earlier))}
    R, H, D, k = case["rows"], case["kv_heads"], case["dim"], case["k"]
    pages = [_pages(v) for v in _lengths(case)]
    q = R * case["heads"] * D * 2
    table = 4 * (max(pages) if case["prefill"] else sum(pages))
    if case["op"] == "block_select":
        boxes = max(pages) if case["prefill"] else sum(pages)
        return {"bytes": boxes * H * (2 * D + 4) + q + table + 4 * R * H * k, "flops": sum(pages) * H * 4 * D}
    token = 2 * (D * BYTES[case["kv"]] + (4 if case["kv"] == "fp8" else 0))
    lens = _lengths(case)
    if not k:
        read = pairs = sum(lens)
    else:
        # the newest page is among them, and ends with the row
        pairs = sum(v if p <= k else (k - 1) * PAGE + v - (p - 1) * PAGE for v, p in zip(lens, pages))
        read = min(pairs, max(lens)) if case["prefill"] else pairs
        table = 4 * R * H * k
    return {"bytes": read * H * token + q + R * case["heads"] * (2 * D + 4) + table,
            "flops": 4 * pairs * case["heads"] * D}


def _exact_slots(case, s):
    new, cached = _new_and_cached(case)
    table, free = s["table"].cpu().tolist(), s["free"].cpu().tolist()
    slots, positions, cu, taken = [], [], [0], 0
    for b, (n, c) in enumerate(zip(new, cached)):
        for p in range(c, c + n):
            if p % PAGE == 0:
                table[b][p // PAGE] = free[taken]
                taken += 1
            slots.append(table[b][p // PAGE] * PAGE + p % PAGE)
            positions.append(p)
        cu.append(cu[-1] + n)
    rest = s["n"] - len(slots)
    return (_int32(table), _int32(slots + [-1] * rest), _int32(positions + [0] * rest),
            _int32([a + b for a, b in zip(new, cached)]), _int32(cu), _int32([taken]))


def _exact_cache(case, s):
    B, n, L = case["requests"], case["tokens"], case["context"]
    pools, scales = [s["k_pool"], s["v_pool"]], [s["k_scale"], s["v_scale"]]
    pools = [p.float().double() for p in pools]
    scales = [None if u is None else u.double() for u in scales]
    for x, pool, scale in zip((s["k"], s["v"]), pools, scales):
        x = x.double()
        page, slot = torch.div(s["slots"], PAGE, rounding_mode="floor").long(), torch.remainder(s["slots"], PAGE).long()
        if scale is not None:
            top = torch.linalg.vector_norm(x, ord=math.inf, dim=-1)
            unit = torch.exp2(torch.ceil(torch.log2(top / 448)))
            unit = torch.where(top > 448 * unit, unit * 2, torch.where(top <= 224 * unit, unit / 2, unit))
            unit = unit.clamp(min=2.0 ** -126)
            v = x / unit[..., None]
            # e4m3: steps of 2^(e - 3), and of 2^-9 below 2^-6; ties to even
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(v / step) * step
            scale[page, :, slot] = unit
        pool[page, :, slot] = x
    keys = pools[0] if scales[0] is None else pools[0] * scales[0][..., None]
    bounds, units = s["bounds"].clone(), s["bound_scale"].double()
    for w in range((L - n) // PAGE, _pages(L)):
        page = s["table"][:, w].long()
        x = keys[page, :, :min(PAGE, L - w * PAGE)]                               # [B, H, tokens, D]
        high, low = x.max(2).values, x.min(2).values
        top = torch.maximum(high, -low).max(-1).values
        unit = torch.exp2(torch.ceil(torch.log2(top / 127)))
        unit = torch.where(top > 127 * unit, unit * 2, torch.where(top <= 63.5 * unit, unit / 2, unit))
        unit = unit.clamp(min=2.0 ** -126)[..., None]
        bounds[page, :, 0] = (high / unit).ceil().to(torch.int8)
        bounds[page, :, 1] = (low / unit).floor().to(torch.int8)
        units[page] = unit[..., 0]
    found = [pools[0], pools[1], bounds, units]
    return found + ([] if scales[0] is None else scales)


def _exact_select(case, s):
    R, H, D, k = case["rows"], case["kv_heads"], case["dim"], case["k"]
    group = case["heads"] // H
    lens = _lengths(case)
    out = torch.full((R, H, k), -1, dtype=torch.int32, device="cuda")
    boxes, scale = s["bounds"].double(), s["bound_scale"].double()
    for j in range(H):
        q = s["q"][:, j * group:(j + 1) * group].double()
        largest = q.abs().reshape(R, -1).max(1).values[:, None, None]
        unit = torch.exp2(torch.floor(torch.log2(largest)) + 1 - GRID)            # 2^-20 of the next power of two
        whole = torch.round(q / unit).to(torch.int64)
        above, below = torch.where(whole > 0, whole, 0).sum(1), torch.where(whole < 0, -whole, 0).sum(1)
        size = torch.maximum(above.max(1).values, below.max(1).values)
        power = torch.ones_like(size)
        for _ in range(24):
            power = torch.where((size + power - 1) // power > 127, power * 2, power)
        above = ((above + power[:, None] - 1) // power[:, None]).double()
        below = ((below + power[:, None] - 1) // power[:, None]).double()
        for r in range(R):
            n = _pages(lens[r])
            page = s["table"][0 if case["prefill"] else r, :n].long()
            score = (boxes[page, j, 0] @ above[r] - boxes[page, j, 1] @ below[r]) * scale[page, j]
            score[0] = score[n - 1] = math.inf
            order = torch.argsort(-score, stable=True)[:k].sort().values
            out[r, j, :order.numel()] = order.to(torch.int32)
    return out


def _exact_attention(case, s):
    R, H, D = case["rows"], case["kv_heads"], case["dim"]
    group = case["heads"] // H
    if (R * H) > 20000:
        return None
    out = torch.zeros((R, case["heads"], D), dtype=torch.float64, device="cuda")
    lse = torch.full((R, case["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    lens = _lengths(case)
    lists = None if s["blocks"] is None else s["blocks"].cpu().tolist()
    for r in range(R):
        row = s["table"][0 if case["prefill"] else r].long()
        for j in range(H):
            blocks = range(_pages(lens[r])) if lists is None else [b for b in lists[r][j] if b >= 0]
            page = row[torch.tensor(list(blocks), device="cuda")]
            k, v = s["k_pool"][page, j].float().double(), s["v_pool"][page, j].float().double()
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][page, j].double()[..., None], v * s["v_scale"][page, j].double()[..., None]
            # pages are in order, so that what lies behind the row's end is the last one's rest
            end = page.numel() * PAGE - (-lens[r]) % PAGE
            k, v = k.flatten(0, 1)[:end], v.flatten(0, 1)[:end]
            heads = slice(j * group, (j + 1) * group)
            logits = (s["q"][r, heads].double() @ k.T) * s["scale"]
            lse[r, heads] = torch.logsumexp(logits, dim=-1)
            out[r, heads] = torch.softmax(logits, dim=-1) @ v
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"request_slots": _exact_slots, "kv_cache": _exact_cache, "block_select": _exact_select,
            "paged_attention": _exact_attention}[case["op"]](case, s)
