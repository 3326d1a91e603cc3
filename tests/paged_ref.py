"""Plain 64-bit references of the operators on the paged cache of keys and values, and builders of
their inputs.  Nothing here uses the library."""
import math

import torch

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp8": torch.float8_e4m3fn}
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}


def pages_of(n):
    return -(-n // PAGE)


# ---- slots from lengths -------------------------------------------------------------

def request_slots(lengths, new, free, table, n):
    """Lists in, lists out: (table, slots, positions, seqlens, cu, used, status)."""
    table = [list(row) for row in table]
    W = len(table[0]) if table else 0
    slots, positions, seqlens, cu, status = [], [], [], [0], 0
    taken = wanted = 0
    for b, (c, m) in enumerate(zip(lengths, new)):
        count = max(m, 0)
        good = c >= 0 and m >= 0 and c + m <= W * PAGE
        ids = {}
        if not good:
            status = max(status, 7)
        else:
            fresh = pages_of(c + m) - pages_of(c)
            if fresh and wanted + fresh > len(free):
                good, status = False, max(status, 6)
            elif fresh:
                taken = wanted + fresh
            for j in range(fresh if good else 0):
                ids[pages_of(c) + j] = free[wanted + j]
                # a page is entered with the token that begins it, if that token has a row
                if cu[-1] + (pages_of(c) + j) * PAGE - c < n:
                    table[b][pages_of(c) + j] = free[wanted + j]
            wanted += fresh
        for i in range(count):
            pos = c + i if good else 0
            page = ids.get(pos // PAGE, table[b][pos // PAGE]) if good else -1
            fits = good and 0 <= page < 2 ** 31 // PAGE - 1
            if good and not fits and cu[-1] + i < n:
                status = max(status, 6)
            slots.append(page * PAGE + pos % PAGE if fits else -1)
            positions.append(pos)
        seqlens.append(c + m if good else 0)
        cu.append(cu[-1] + count)
    if len(slots) > n:
        status = max(status, 7)
    rest = max(0, n - len(slots))
    return table, (slots + [-1] * rest)[:n], (positions + [0] * rest)[:n], seqlens, cu, taken, status


# ---- the cache ----------------------------------------------------------------------

def scale_of(top, most=448.0):
    """2^e, the smallest e >= -126 with top <= most * 2^e (a float)."""
    if top == 0:
        return 2.0 ** -126
    e = math.ceil(math.log2(top / most))
    while top > most * 2.0 ** e:
        e += 1
    while top <= most * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -126)


def quantise(x):
    """x [..., D] -> (e4m3 codes, fp32 scale [...]) as the store's definition has them."""
    flat = x.double().reshape(-1, x.shape[-1])
    top = torch.where(flat.isfinite(), flat.abs(), 0.0).amax(-1)
    scale = torch.tensor([scale_of(v) for v in top.tolist()], dtype=torch.float64)
    y = flat / scale[:, None]
    y = torch.where(y.isnan(), y, y.clamp(-448, 448))
    codes = y.float().to(torch.float8_e4m3fn)          # the quotient is exact in 32 bits (normal scales)
    return codes.reshape(x.shape), scale.float().reshape(x.shape[:-1])


def box(keys):
    """Box of keys [tokens, D] (64 bits): (codes [2, D] as ints, scale)."""
    most = float(torch.finfo(torch.float32).max)
    k = keys.clamp(-most, most)
    high = torch.where(k.isnan(), -math.inf, k).amax(0)
    low = torch.where(k.isnan(), math.inf, k).amin(0)
    none = low > high
    high, low = torch.where(none, 0.0, high), torch.where(none, 0.0, low)
    unit = scale_of(float(torch.maximum(high.abs(), low.abs()).max()), 127.0)
    return torch.stack([torch.ceil(high / unit), torch.floor(low / unit)]).to(torch.int8), unit


# ---- selection ------------------------------------------------------------------------

def select(q, boxes, scale, k, first, last):
    """q [group, D], boxes [n, 2, D] ints, scale [n] -> ascending list of at most k places."""
    n = boxes.shape[0]
    if n <= k:
        return list(range(n))
    most = float(torch.finfo(torch.float32).max)
    q = torch.nan_to_num(q.double(), nan=0.0, posinf=most, neginf=-most).clamp(-most, most)
    top = float(q.abs().max())
    x = math.frexp(top)[1]
    whole = torch.round(q * 2.0 ** (20 - x))
    above, below = whole.clamp(min=0).sum(0), (-whole).clamp(min=0).sum(0)
    size, s = max(float(above.max()), float(below.max())), 0
    while size > 127 * 2 ** s:
        s += 1
    p, m = torch.ceil(above / 2 ** s), torch.ceil(below / 2 ** s)
    dot = boxes[:, 0].double() @ p - boxes[:, 1].double() @ m
    score = (dot * scale.double()).clamp(-most, most).tolist()
    forced = [i < first or i >= n - last for i in range(n)]
    order = sorted(range(n), key=lambda i: (not forced[i], 0.0 if forced[i] else -score[i], i))
    return sorted(order[:k])


# ---- attention ------------------------------------------------------------------------

def attention_row(q, k, v, scale, kv, out_type):
    """q [Hq, D], k and v [T, Hkv, D], 64 bits -> (out, lse, and what they may be off).

    The bounds count: the result's rounding; the weights' rounding to the cache's type (fp8: fp16),
    2^-25 of the largest where fp16 leaves its normal numbers; scores and sums in fp32 (tensor
    cores: twice a rounding per addition); exponentials to 2^-21.
    """
    Hq, T, group = q.shape[0], k.shape[0], q.shape[0] // k.shape[1]
    if T == 0:
        return (torch.zeros_like(q), q.new_full((Hq,), -math.inf), torch.zeros_like(q), q.new_zeros(Hq))
    kh, vh = k.repeat_interleave(group, 1).transpose(0, 1), v.repeat_interleave(group, 1).transpose(0, 1)
    s = (kh @ q[:, :, None])[..., 0] * scale                              # [Hq, T]
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    out = (p[:, None] @ vh)[:, 0]
    size = (p[:, None] @ vh.abs())[:, 0]
    f32 = 2.0 ** -24
    ds = (2 * (q.shape[1] + 8) * f32 * ((kh.abs() @ q.abs()[:, :, None])[..., 0] * abs(scale)).amax(-1)
          + 4 * f32 * s.abs().amax(-1) + 2.0 ** -21)
    weight = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    tiny = 0.0 if kv == "bf16" else 2.0 ** -25
    sums = 2 * (T / 8 + 64) * f32
    bound = (HALF[out_type] * out.abs() + (1 + 2.0 ** -7) * (weight + 2 * ds[:, None] + sums) * size
             + T * tiny * p.amax(-1)[:, None] * vh.abs().amax(1))
    if out_type == torch.float16:
        bound = bound + 2.0 ** -25
    return out, lse, bound, ds + sums + 4 * f32 * (lse.abs() + 1)


class Pools:
    """Pools of keys and values with NaN wherever no token is, in the page layout that `layout` names."""

    def __init__(self, pages, heads, dim, kv, layout="head"):
        self.kv, self.heads, self.dim, dtype = kv, heads, dim, TYPES[kv]

        def full(*shape):
            if kv == "fp8":
                return torch.full(shape, 0x7f, dtype=torch.uint8).view(dtype)
            return torch.full(shape, math.nan, dtype=dtype)
        if layout == "head":
            self.k, self.v = (full(pages, heads, PAGE, dim).transpose(1, 2) for _ in range(2))
        elif layout == "token":
            self.k, self.v = (full(pages, PAGE, heads, dim) for _ in range(2))
        elif layout == "both":              # keys and values of a page side by side
            both = full(pages, 2, heads, PAGE, dim)
            self.k, self.v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
        else:                                # "wide": every dimension longer than what is used
            wide = full(pages * 2, PAGE, heads + 1, dim + 32)
            self.k = wide[::2, :, :heads, :dim]
            self.v = full(pages, PAGE, heads, dim * 2)[..., dim:]
        self.k_scale = self.v_scale = None
        if kv == "fp8":
            self.k_scale = torch.full((pages, heads, PAGE), math.nan)
            self.v_scale = torch.full((pages, heads, PAGE), math.nan)

    def put(self, page, slot, k, v):
        """Tokens k, v [n, Hkv, D] (any float type) into their places."""
        for x, pool, scale in ((k, self.k, self.k_scale), (v, self.v, self.v_scale)):
            if scale is None:
                pool[page, slot] = x.to(pool.dtype)
            else:
                codes, s = quantise(x)
                bytes_of(pool)[page, slot] = codes.view(torch.uint8)
                scale[page, :, slot] = s

    def get(self, page, slot):
        """Keys and values [n, Hkv, D] in 64 bits."""
        found = []
        for pool, scale in ((self.k, self.k_scale), (self.v, self.v_scale)):
            if scale is None:
                found.append(pool[page, slot].double())
            else:
                x = bytes_of(pool)[page, slot].contiguous().view(torch.float8_e4m3fn).float().double()
                found.append(x * scale[page, :, slot].double()[..., None])
        return found

    def cuda(self):
        """(k, v, k_scale, v_scale) on the GPU with the same strides."""
        done, seen = [], {}
        for x in (self.k, self.v):
            base = x._base if x._base is not None else x
            while base._base is not None:
                base = base._base
            if base.data_ptr() not in seen:
                seen[base.data_ptr()] = base.cuda().reshape(-1).view(x.dtype)
            done.append(seen[base.data_ptr()].as_strided(x.shape, x.stride(), x.storage_offset()))
        return done + [None if s is None else s.cuda() for s in (self.k_scale, self.v_scale)]


def bytes_of(x):
    """A float8 tensor as bytes (indexing and copies that every device has)."""
    return x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
