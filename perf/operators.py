"""Performance cases of the operators around sparse latent attention.

Three operators of a sparse-attention decoder layer, each reached through
``sparse_attention_paged_gb300``:

``qk_norm_rope``
    Per-head normalisation of queries and keys with the position rotation in
    the same pass.
``latent_cache``
    The paged cache of one latent vector (512 values) and one rotated key
    part (64 values) per token: normalise, rotate and quantise new tokens into
    their pages (``latent_store``), and read a range of tokens back
    (``latent_load``).
``latent_attention``
    Attention of H query heads over the cached tokens of a row, in the
    absorbed form: scores against all 576 values, outputs the weighted sum of
    the 512 latent ones.  Either every position below the row's length is
    read, or the positions of a selection list.

``own`` chooses between the plain form (elementary torch operations in 32
bits, rounded once at the end) and the library's calls.
"""
import math

import torch

own = False

PAGE = 64       # positions per cache page
LATENT = 512    # latent values per token
ROPE = 64       # rotated values per token
GROUP = 128     # latent values that share one scale
BASE = 10000.0  # base of the rotation's frequencies
EPS = 1e-6

# bytes of one cached token: bf16 values, or e4m3 codes + 4 scales + bf16 rotated part
TOKEN_BYTES = {"bf16": 2 * (LATENT + ROPE), "fp8": LATENT + 4 * (LATENT // GROUP) + 2 * ROPE}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _norm(name, tokens, q_heads, k_heads, dim, rot, offset, interleaved, norm, dtype):
    return {"name": name, "op": "qk_norm_rope", "tokens": tokens, "q_heads": q_heads,
            "k_heads": k_heads, "dim": dim, "rot": rot, "offset": offset,
            "interleaved": interleaved, "norm": norm, "dtype": dtype, "max_pos": 131072}


def _cache(name, requests, tokens, context, kv, interleaved):
    return {"name": name, "op": "latent_cache", "requests": requests, "tokens": tokens,
            "context": context, "kv": kv, "interleaved": interleaved, "max_pos": 131072}


def _attention(name, rows, heads, kv, k, min_len, max_len, prefill):
    return {"name": name, "op": "latent_attention", "rows": rows, "heads": heads, "kv": kv,
            "k": k, "min_len": min_len, "max_len": max_len, "prefill": prefill}


def listed():
    return [
        # one decode step of 64 requests: the indexer's 64 query heads and its one key head
        _norm("norm_rope_decode_64", 64, 64, 1, 128, 64, 0, False, "layer", "bf16"),
        # a prefill chunk of 4,096 tokens, the same heads
        _norm("norm_rope_prefill_4096", 4096, 64, 1, 128, 64, 0, False, "layer", "bf16"),
        # grouped heads of another width, interleaved pairs, an odd number of tokens
        _norm("norm_rope_fp16_1337", 1337, 24, 8, 192, 64, 128, True, "rms", "fp16"),
        # one decode step of 64 short requests: one token each written, the contexts read back
        _cache("cache_fp8_decode_64", 64, 1, 65, "fp8", True),
        # a prefill of 22,528 tokens written, and the whole context read back
        _cache("cache_fp8_prefill_22528", 1, 22528, 22528, "fp8", True),
        # a batch of ragged chunks over earlier context, bf16 cache
        _cache("cache_bf16_ragged_5x997", 5, 997, 5003, "bf16", False),
        # the smallest call: one request, a short selection list, few heads of a split model
        _attention("attn_sparse_fp8_b1_k512", 1, 16, "fp8", 512, 4096, 4096, False),
        # decode over selected positions, long bf16 contexts
        _attention("attn_sparse_bf16_b64_k2048", 64, 64, "bf16", 2048, 4096, 131072, False),
        # decode over every position, fp8 cache, lengths log-uniform
        _attention("attn_dense_fp8_b64", 64, 64, "fp8", 0, 512, 32768, False),
        # decode of one long request with twice the heads
        _attention("attn_dense_bf16_b1_131072", 1, 128, "bf16", 0, 131072, 131072, False),
        # odd sizes: 37 heads, a list that ends inside a tile, lengths from one token
        _attention("attn_sparse_fp8_b19_k777", 19, 37, "fp8", 777, 1, 9001, False),
        # a prefill chunk over a shared context, every query token with its own selection
        _attention("attn_prefill_fp8_1024_k2048", 1024, 64, "fp8", 2048, 0, 22528, True),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["qk_norm_rope", "latent_cache", "latent_attention", "latent_attention"])
    if kind == "qk_norm_rope":
        dim = rng.choice([64, 96, 128, 192, 256])
        rot = rng.choice([r for r in (32, 64, 128) if r <= dim])
        case = _norm("", _log_int(rng, 1, 4096), rng.randint(1, 64), rng.randint(1, 8), dim, rot,
                     rng.choice([0, dim - rot]), rng.random() < 0.5, rng.choice(["layer", "rms"]),
                     rng.choice(["bf16", "fp16", "fp32"]))
        if case["tokens"] * case["q_heads"] * dim > 4096 * 64 * 128:
            case["tokens"] = 4096 * 64 * 128 // (case["q_heads"] * dim)
    elif kind == "latent_cache":
        requests = _log_int(rng, 1, 64)
        context = _log_int(rng, 1, 22528 // requests)
        case = _cache("", requests, _log_int(rng, 1, context), context, rng.choice(["fp8", "bf16"]),
                      rng.random() < 0.5)
    elif rng.random() < 0.25:
        # prefill: consecutive query tokens over one shared context
        rows = _log_int(rng, 2, 1024)
        context = rows + _log_int(rng, 1, 22528 - rows)
        case = _attention("", rows, rng.choice([16, 32, 64]), rng.choice(["fp8", "bf16"]),
                          _log_int(rng, 1, 2048), 0, context, True)
    else:
        rows = _log_int(rng, 1, 64)
        k = rng.choice([0, 0, _log_int(rng, 1, 2048), _log_int(rng, 1, 2048)])
        top = _log_int(rng, 1, min(131072, 2097152 // rows))
        case = _attention("", rows, rng.choice([1, 8, 16, 32, 48, 64, 100, 128]),
                          rng.choice(["fp8", "bf16"]), k, max(1, top // 32), top, False)
    del case["name"]
    return case


def _lengths(case):
    """Lengths of the rows: the causal limits of a prefill, else log-uniform (even quantiles)."""
    rows, low, high = case["rows"], case["min_len"], case["max_len"]
    if case["prefill"]:
        return [high - rows + 1 + i for i in range(rows)]
    if rows == 1:
        return [high]
    ratio = math.log(high / low)
    return [min(high, int(low * math.exp(ratio * i / (rows - 1)))) for i in range(rows)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _table(max_pos, rot):
    """fp32 [max_pos, rot]: rot/2 cosines, then rot/2 sines, of the angles of each position."""
    freq = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    angle = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], dim=1).float()


def _layout(kv):
    """Byte offsets of a page's parts: (latent, rotated part, scales, page bytes)."""
    if kv == "bf16":
        return 0, 2 * LATENT, None, PAGE * TOKEN_BYTES["bf16"]
    codes, rope = PAGE * LATENT, PAGE * ROPE * 2
    return 0, codes, codes + rope, PAGE * TOKEN_BYTES["fp8"]


def _cache_views(pool, kv):
    """Views of a pool [pages, page bytes]: latent codes or values, rotated part, scales."""
    pages = pool.shape[0]
    if kv == "bf16":
        v = pool.view(torch.bfloat16).view(pages, PAGE, LATENT + ROPE)
        return v[..., :LATENT], v[..., LATENT:], None
    _, rope_at, scale_at, end = _layout(kv)
    codes = pool[:, :rope_at].view(torch.float8_e4m3fn).view(pages, PAGE, LATENT)
    rope = pool[:, rope_at:scale_at].view(torch.bfloat16).view(pages, PAGE, ROPE)
    scale = pool[:, scale_at:end].view(torch.float32).view(pages, PAGE, LATENT // GROUP)
    return codes, rope, scale


def _scales(groups):
    """The smallest power of two that brings each group's largest magnitude to at most 448."""
    top = groups.abs().amax(dim=-1)
    mantissa, exponent = torch.frexp(top)                 # top = mantissa * 2^exponent, mantissa in [0.5, 1)
    e = torch.where(mantissa <= 0.875, exponent - 9, exponent - 8).clamp(-126, 127)
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e), torch.ones_like(top))


def _fill_pool(pages, kv, g):
    """A pool of random tokens, some pages at a time."""
    pool = torch.empty((pages, _layout(kv)[3]), dtype=torch.uint8, device="cuda")
    latent, rope, scale = _cache_views(pool, kv)
    for at in range(0, pages, 4096):
        n = min(4096, pages - at)
        if kv == "bf16":
            latent[at:at + n] = torch.randn((n, PAGE, LATENT), generator=g, device="cuda", dtype=torch.bfloat16)
        else:
            x = torch.randn((n, PAGE, LATENT // GROUP, GROUP), generator=g, device="cuda")
            s = _scales(x)
            scale[at:at + n] = s
            latent[at:at + n] = (x / s[..., None]).view(n, PAGE, LATENT).to(torch.float8_e4m3fn)
        rope[at:at + n] = torch.randn((n, PAGE, ROPE), generator=g, device="cuda", dtype=torch.bfloat16)
    return pool


def _prepare_norm(case, g):
    T, D, dtype = case["tokens"], case["dim"], TYPES[case["dtype"]]
    hq, hk = case["q_heads"], case["k_heads"]
    # one projection's output, heads side by side: queries, then keys
    x = torch.randn((T, hq + hk, D), generator=g, device="cuda").to(dtype)
    layer = case["norm"] == "layer"
    weight = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    bias = [0.1 * torch.randn(D, generator=g, device="cuda") if layer else None for _ in range(2)]
    y = torch.empty_like(x)
    return {"q": x[:, :hq], "k": x[:, hq:], "weight": weight, "bias": bias,
            "positions": torch.randint(0, case["max_pos"], (T,), generator=g, device="cuda", dtype=torch.int32),
            "table": _table(case["max_pos"], case["rot"]), "q_out": y[:, :hq], "k_out": y[:, hq:]}


def _prepare_cache(case, g):
    B, n, L = case["requests"], case["tokens"], case["context"]
    W = (L + PAGE - 1) // PAGE
    table = torch.randperm(B * W, generator=g, device="cuda").to(torch.int32).view(B, W)
    # the last n of each request's L positions are new
    pos = torch.arange(L - n, L, device="cuda").expand(B, n)
    slots = table.long().gather(1, pos // PAGE) * PAGE + pos % PAGE
    magnitude = torch.exp(0.5 * torch.randn((B * n, 1), generator=g, device="cuda"))
    x = torch.randn((B * n, LATENT + ROPE), generator=g, device="cuda") * magnitude
    return {"x": x.to(torch.bfloat16), "weight": 1 + 0.1 * torch.randn(LATENT, generator=g, device="cuda"),
            "positions": pos.reshape(-1).to(torch.int32).contiguous(),
            "table": _table(case["max_pos"], ROPE),
            "slots": slots.reshape(-1).to(torch.int32), "pool": _fill_pool(B * W, case["kv"], g),
            "block_table": table, "starts": torch.zeros(B, dtype=torch.int32, device="cuda"),
            "cu": torch.arange(0, (B + 1) * L, L, device="cuda", dtype=torch.int32),
            "out": torch.empty((B * L, LATENT + ROPE), dtype=torch.bfloat16, device="cuda")}


def _prepare_attention(case, g):
    R, H, k = case["rows"], case["heads"], case["k"]
    lens = _lengths(case)
    W = (max(lens) + PAGE - 1) // PAGE
    seqlens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    if case["prefill"]:
        pages = W
        table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).view(1, W)
    else:
        used = (seqlens.long() + PAGE - 1) // PAGE
        pages = sum((v + PAGE - 1) // PAGE for v in lens)
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        at = (used.cumsum(0) - used)[:, None] + torch.arange(W, device="cuda")
        table = torch.where(torch.arange(W, device="cuda") < used[:, None],
                            perm[at.clamp(max=pages - 1)], torch.zeros_like(perm[:1])).contiguous()
    idx = None
    if k:
        n = max(k, max(lens))
        keys = torch.rand((R, n), generator=g, device="cuda")
        keys.masked_fill_(torch.arange(n, device="cuda") >= seqlens[:, None], -1.0)
        best, where = keys.topk(k, dim=1)
        where = torch.where(best >= 0, where, n).sort(dim=1).values
        idx = torch.where(where < n, where, -1).to(torch.int32)
    q = torch.randn((R, H, LATENT + ROPE), generator=g, device="cuda").to(torch.bfloat16)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return {"q_latent": q[..., :LATENT].contiguous(), "q_rope": q[..., LATENT:].contiguous(),
            "pool": _fill_pool(pages, case["kv"], g), "block_table": table, "seqlens": seqlens,
            "idx": idx, "scale": 192 ** -0.5,
            "out": torch.empty((R, H, LATENT), dtype=torch.bfloat16, device="cuda"),
            "lse": torch.empty((R, H), dtype=torch.float32, device="cuda"),
            # two partial rows per SM (64 heads, 512 sums and two statistics each), and a split record
            "workspace": torch.empty(sms * (2 * 64 * 514 + 64), dtype=torch.float32, device="cuda")}


def prepare(case, seed):
    g = _generator(seed)
    make = {"qk_norm_rope": _prepare_norm, "latent_cache": _prepare_cache,
            "latent_attention": _prepare_attention}[case["op"]]
    return {"case": dict(case), **make(case, g)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _rotate(x, table, positions, interleaved):
    """Rotation of the pairs of x [T, heads, rot] by the angles of each token's position."""
    half = x.shape[-1] // 2
    row = table[positions.long()][:, None]
    cos, sin = row[..., :half], row[..., half:]
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)


def _plain_norm_rope(s):
    case, done = s["case"], []
    at, end = case["offset"], case["offset"] + case["rot"]
    for x, w, b in ((s["q"], s["weight"][0], s["bias"][0]), (s["k"], s["weight"][1], s["bias"][1])):
        y = x.float()
        if case["norm"] == "layer":
            y = y - y.mean(-1, keepdim=True)
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w
        y = y if b is None else y + b
        y = torch.cat([y[..., :at], _rotate(y[..., at:end], s["table"], s["positions"], case["interleaved"]),
                       y[..., end:]], dim=-1)
        done.append(y.to(x.dtype))
    return done


def _plain_cache(s):
    case, kv = s["case"], s["case"]["kv"]
    latent, rope, scale = _cache_views(s["pool"], kv)
    x = s["x"].float()
    c = x[:, :LATENT]
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"]
    r = _rotate(x[:, None, LATENT:], s["table"], s["positions"], case["interleaved"])[:, 0]
    page, slot = s["slots"].long() // PAGE, s["slots"].long() % PAGE
    rope[page, slot] = r.to(torch.bfloat16)
    if kv == "bf16":
        latent[page, slot] = c.to(torch.bfloat16)
    else:
        groups = c.view(-1, LATENT // GROUP, GROUP)
        e = _scales(groups)
        scale[page, slot] = e
        codes = (groups / e[..., None]).view(-1, LATENT).to(torch.float8_e4m3fn)
        latent.view(torch.uint8)[page, slot] = codes.view(torch.uint8)
    page, slot = _token_slots(s["block_table"], case["context"])
    return _tokens(latent, rope, scale, page, slot).to(torch.bfloat16)


def _token_slots(table, length):
    """Page and slot of every position below `length` of every request, requests in order."""
    pos = torch.arange(length, device=table.device).expand(table.shape[0], length)
    return table.long().gather(1, pos // PAGE).reshape(-1), (pos % PAGE).reshape(-1)


def _tokens(latent, rope, scale, page, slot):
    """The cached tokens at (page, slot) in 32 bits: latent values, then the rotated part."""
    if scale is None:
        c = latent[page, slot].float()
    else:
        c = latent.view(torch.uint8)[page, slot].view(torch.float8_e4m3fn).float()
        c = c * scale[page, slot].repeat_interleave(GROUP, dim=-1)
    return torch.cat([c, rope[page, slot].float()], dim=-1)


def _plain_attention(s):
    case = s["case"]
    R, table = case["rows"], s["block_table"].long()
    seqlens = s["seqlens"].long()[:, None]
    if s["idx"] is None:
        pos = torch.arange(table.shape[1] * PAGE, device=table.device).expand(R, -1)
    else:
        pos = s["idx"].long()
    valid = (pos >= 0) & (pos < seqlens)
    pos = torch.where(valid, pos, 0)
    page = table.expand(R, -1).gather(1, pos // PAGE)
    kv = _tokens(*_cache_views(s["pool"], case["kv"]), page, pos % PAGE)          # [R, K, 576]
    kv = torch.where(valid[..., None], kv, 0.0)
    q = torch.cat([s["q_latent"], s["q_rope"]], dim=-1).float()
    score = torch.bmm(q, kv.transpose(1, 2)) * s["scale"]                          # [R, H, K]
    score = torch.where(valid[:, None], score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p, kv[..., :LATENT]) / torch.where(total > 0, total, 1.0)
    return out.to(torch.bfloat16), (top + torch.log(total)).squeeze(-1)


def _own_norm_rope(s):
    import sparse_attention_paged_gb300 as lib
    case = s["case"]
    lib.qk_norm_rope(s["q"], s["k"], s["positions"], s["table"], rot_dims=case["rot"],
                     rot_offset=case["offset"], interleaved=case["interleaved"],
                     norm=lib.NORM_LAYER if case["norm"] == "layer" else lib.NORM_RMS,
                     q_weight=s["weight"][0], k_weight=s["weight"][1], q_bias=s["bias"][0],
                     k_bias=s["bias"][1], eps=EPS, q_out=s["q_out"], k_out=s["k_out"])
    return [s["q_out"], s["k_out"]]


def _own_cache(s):
    import sparse_attention_paged_gb300 as lib
    case = s["case"]
    kv = lib.KV_BF16 if case["kv"] == "bf16" else lib.KV_FP8_E4M3
    lib.latent_store(s["x"][:, :LATENT], s["x"][:, LATENT:], s["slots"], s["pool"], kv,
                     norm_weight=s["weight"], eps=EPS, positions=s["positions"],
                     rope_table=s["table"], interleaved=case["interleaved"])
    return lib.latent_load(s["pool"], kv, s["block_table"], s["cu"], s["out"].shape[0],
                           starts=s["starts"], out=s["out"])


def _own_attention(s):
    import sparse_attention_paged_gb300 as lib
    case = s["case"]
    kv = lib.KV_BF16 if case["kv"] == "bf16" else lib.KV_FP8_E4M3
    lib.latent_attention(s["q_latent"], s["q_rope"], s["pool"], kv, s["block_table"], s["seqlens"],
                         s["scale"], idx=s["idx"], out=s["out"], lse=s["lse"],
                         workspace=s["workspace"])
    return s["out"], s["lse"]


def run(state):
    form = {"qk_norm_rope": (_plain_norm_rope, _own_norm_rope),
            "latent_cache": (_plain_cache, _own_cache),
            "latent_attention": (_plain_attention, _own_attention)}[state["case"]["op"]]
    return form[1 if own else 0](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its result in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "qk_norm_rope":
        values = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"]
        angles = min(case["tokens"], case["max_pos"]) * case["rot"] * 4
        return {"bytes": 2 * values * BYTES[case["dtype"]] + angles + case["tokens"] * 4,
                "flops": values * 8}
    if case["op"] == "latent_cache":
        new, all_ = case["requests"] * case["tokens"], case["requests"] * case["context"]
        token = TOKEN_BYTES[case["kv"]]
        written = new * (2 * (LATENT + ROPE) + ROPE * 4 + 8 + token)
        return {"bytes": written + all_ * (token + 2 * (LATENT + ROPE)),
                "flops": new * LATENT * 8 + all_ * LATENT}
    lens, k = _lengths(case), case["k"]
    read = [min(v, k) if k else v for v in lens]
    pairs = sum(read)
    if case["prefill"]:
        # the tokens that any row selects: at most the whole context, each once
        tokens = min(pairs, case["max_len"])
    else:
        tokens = pairs
    q = case["rows"] * case["heads"] * (LATENT + ROPE) * 2
    out = case["rows"] * case["heads"] * (LATENT * 2 + 4)
    return {"bytes": tokens * TOKEN_BYTES[case["kv"]] + q + out + (4 * pairs if k else 0),
            "flops": 2 * pairs * case["heads"] * (2 * LATENT + ROPE)}


def _angles64(case, positions, rot):
    freq = torch.tensor([BASE ** (-2 * i / rot) for i in range(rot // 2)], dtype=torch.float64, device="cuda")
    return positions.double()[:, None] * freq


def _turn64(x, angle, interleaved):
    """Pairs of x [..., rot] as complex numbers, turned by `angle` [..., rot / 2]."""
    pairs = x.unflatten(-1, (-1, 2)) if interleaved else x.unflatten(-1, (2, -1)).transpose(-1, -2)
    z = torch.view_as_complex(pairs.contiguous()) * torch.polar(torch.ones_like(angle), angle)
    z = torch.view_as_real(z)
    return z.flatten(-2) if interleaved else z.transpose(-1, -2).flatten(-2)


def _exact_norm_rope(case, s):
    angle = _angles64(case, s["positions"], case["rot"])[:, None]
    found = []
    for x, w, b in zip((s["q"], s["k"]), s["weight"], s["bias"]):
        y = x.double()
        if case["norm"] == "layer":
            variance, mean = torch.var_mean(y, dim=-1, correction=0, keepdim=True)
            y = (y - mean) / torch.sqrt(variance + EPS)
        else:
            y = y / torch.sqrt(torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / case["dim"] + EPS)
        y = y * w.double()
        if b is not None:
            y = y + b.double()
        part = slice(case["offset"], case["offset"] + case["rot"])
        y[..., part] = _turn64(y[..., part].clone(), angle.expand(-1, y.shape[1], -1), case["interleaved"])
        found.append(y)
    return found


def _exact_cache(case, s):
    x = s["x"].double()
    c = x[:, :LATENT]
    c = c / torch.sqrt(torch.linalg.vector_norm(c, dim=-1, keepdim=True) ** 2 / LATENT + EPS) * s["weight"].double()
    r = _turn64(x[:, LATENT:].clone(), _angles64(case, s["positions"], ROPE), case["interleaved"])
    B, n, L = case["requests"], case["tokens"], case["context"]
    out = torch.empty((B, L, LATENT + ROPE), dtype=torch.float64, device="cuda")
    for b in range(B):
        for w in range(s["block_table"].shape[1]):
            end = min(PAGE, L - w * PAGE)
            out[b, w * PAGE:w * PAGE + end] = _page64(s["pool"], case["kv"], int(s["block_table"][b, w]))[:end]
    # a new token holds the normed latent and the turned part, to the cache's precision
    if case["kv"] == "fp8":
        for at in range(0, LATENT, GROUP):
            part = c[:, at:at + GROUP]
            top = part.abs().amax(-1, keepdim=True)
            unit = torch.exp2(torch.ceil(torch.log2(top / 448)))
            unit = torch.where(top > 448 * unit, unit * 2, torch.where(top <= 224 * unit, unit / 2, unit))
            v = part / unit
            # e4m3: steps of 2^(e - 3), and of 2^-9 below 2^-6; ties to even
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            c[:, at:at + GROUP] = torch.round(v / step) * step * unit
    out[:, L - n:, :LATENT] = c.view(B, n, LATENT)
    out[:, L - n:, LATENT:] = r.view(B, n, ROPE)
    return out.view(B * L, LATENT + ROPE)


def _page64(pool, kv, page):
    """One page [64, 576] in 64 bits."""
    raw = pool[page]
    if kv == "bf16":
        return raw.view(torch.bfloat16).double().view(PAGE, LATENT + ROPE)
    a, b = PAGE * LATENT, PAGE * (LATENT + 2 * ROPE)
    codes = raw[:a].view(torch.float8_e4m3fn).float().double().view(PAGE, LATENT // GROUP, GROUP)
    unit = raw[b:].view(torch.float32).double().view(PAGE, LATENT // GROUP, 1)
    rope = raw[a:b].view(torch.bfloat16).double().view(PAGE, ROPE)
    return torch.cat([(codes * unit).view(PAGE, LATENT), rope], dim=1)


def _exact_attention(case, s):
    R, H = case["rows"], case["heads"]
    out = torch.zeros((R, H, LATENT), dtype=torch.float64, device="cuda")
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device="cuda")
    lens, pool, kv = _lengths(case), s["pool"], case["kv"]
    stride = TOKEN_BYTES[kv]
    for r in range(R):
        row = s["block_table"][0 if case["prefill"] else r].long()
        t = torch.arange(lens[r], device="cuda")
        if s["idx"] is not None:
            t = s["idx"][r].long()
            t = t[(t >= 0) & (t < lens[r])]
        if not t.numel():
            continue
        page, slot = row[t // PAGE], t % PAGE
        if kv == "bf16":
            x = pool.view(-1, stride)[page * PAGE + slot].view(torch.bfloat16).double()
        else:
            c = pool[:, :PAGE * LATENT].view(-1, PAGE, LATENT)[page, slot].view(torch.float8_e4m3fn).float().double()
            u = pool[:, PAGE * (LATENT + 2 * ROPE):].view(torch.float32).view(-1, PAGE, 4)[page, slot].double()
            k = pool[:, PAGE * LATENT:PAGE * (LATENT + 2 * ROPE)].view(torch.bfloat16).view(-1, PAGE, ROPE)[page, slot]
            x = torch.cat([(c.view(-1, 4, GROUP) * u[..., None]).flatten(1), k.double()], dim=1)
        q = torch.cat([s["q_latent"][r], s["q_rope"][r]], dim=-1).double()
        logits = (q @ x.T) * s["scale"]
        lse[r] = torch.logsumexp(logits, dim=-1)
        out[r] = torch.exp(logits - lse[r][:, None]) @ x[:, :LATENT]
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    return {"qk_norm_rope": _exact_norm_rope, "latent_cache": _exact_cache,
            "latent_attention": _exact_attention}[case["op"]](case, s)
