"""Plain 64-bit references of the operators around the sparse attention, and
builders of their inputs.  Nothing here uses the library."""
import math

import numpy as np
import torch

LATENT, ROPE, GROUP, PAGE = 512, 64, 128, 64
KV_FP8, KV_BF16 = 0, 1
PAGE_BYTES = {KV_FP8: 41984, KV_BF16: 73728}


def angles(positions, rot, base=10000.0):
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return positions.double()[:, None] * f


def rotate(x, angle, interleaved):
    """x [..., rot] in 64 bits, angle broadcastable to [..., rot / 2]."""
    half = x.shape[-1] // 2
    c, s = angle.cos(), angle.sin()
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :half], x[..., half:])
    y, z = a * c - b * s, b * c + a * s
    if interleaved:
        return torch.stack([y, z], -1).reshape(x.shape)
    return torch.cat([y, z], -1)


def norm(x, kind, weight, bias, eps):
    """kind: 0 none, 1 rms, 2 layer; 64 bits."""
    if kind == 0:
        return x
    if kind == 2:
        x = x - x.mean(-1, keepdim=True)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    return y if bias is None else y + bias.double()


def norm_rope(x, kind, weight, bias, eps, positions, rot, offset, interleaved):
    y = norm(x.double(), kind, weight, bias, eps)
    if positions is not None:
        y = y.clone()
        part = slice(offset, offset + rot)
        y[..., part] = rotate(y[..., part], angles(positions, rot)[:, None], interleaved)
    return y


def scale_of(top):
    """The fp8 scale of a group whose largest finite magnitude is `top` (a float)."""
    if top == 0:
        return 1.0
    e = math.ceil(math.log2(top / 448.0))
    while top > 448.0 * 2.0 ** e:
        e += 1
    while top <= 448.0 * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(e, -126)


def quantise(c):
    """c [n, 512] float64 -> codes uint8 [n, 512], scales float32 [n, 4] by the definition."""
    n = c.shape[0]
    groups = c.view(n, 4, GROUP)
    finite = torch.where(torch.isfinite(groups), groups.abs(), torch.zeros_like(groups))
    scales = torch.tensor([[scale_of(float(v)) for v in row] for row in finite.amax(-1)],
                          dtype=torch.float64).view(n, 4)
    v = (groups / scales[..., None]).clamp(-448, 448)          # clamp keeps NaN
    codes = v.float().to(torch.float8_e4m3fn).view(torch.uint8).reshape(n, LATENT)
    return codes, scales.float()


def page_views(pool, kv):
    """(latent codes or values, rotated part, scales or None) of a CPU pool [pages, bytes]."""
    n = pool.shape[0]
    if kv == KV_BF16:
        v = pool[:, :73728].view(torch.bfloat16).view(n, PAGE, 576)
        return v[..., :LATENT], v[..., LATENT:], None
    return (pool[:, :32768].view(n, PAGE, LATENT),
            pool[:, 32768:40960].view(torch.bfloat16).view(n, PAGE, ROPE),
            pool[:, 40960:41984].view(torch.float32).view(n, PAGE, 4))


def tokens(pool, kv, page, slot):
    """[n, 576] in 64 bits."""
    latent, rope, scale = page_views(pool, kv)
    r = rope[page, slot].double()
    if kv == KV_BF16:
        return torch.cat([latent[page, slot].double(), r], -1)
    c = latent[page, slot].contiguous().view(torch.float8_e4m3fn).float().double()
    return torch.cat([c * scale[page, slot].double().repeat_interleave(GROUP, -1), r], -1)


def random_pool(pages, kv, g, stride=None):
    """A CPU pool of random tokens; `stride` > the page's bytes leaves a poisoned gap."""
    stride = stride or PAGE_BYTES[kv]
    pool = torch.full((pages, stride), 0x7f, dtype=torch.uint8)
    rope = torch.randn((pages, PAGE, ROPE), generator=g).to(torch.bfloat16)
    c = torch.randn((pages * PAGE, LATENT), generator=g)
    if kv == KV_BF16:
        v = torch.cat([c.view(pages, PAGE, LATENT).to(torch.bfloat16), rope], -1)
        pool[:, :73728] = v.contiguous().view(torch.uint8).view(pages, -1)
        return pool
    codes, scales = quantise_fast(c)
    pool[:, :32768] = codes.view(pages, -1)
    pool[:, 32768:40960] = rope.contiguous().view(torch.uint8).view(pages, -1)
    pool[:, 40960:41984] = scales.view(torch.uint8).view(pages, -1)
    return pool


def quantise_fast(c):
    top = c.view(-1, 4, GROUP).abs().amax(-1)
    s = torch.exp2(torch.ceil(torch.log2(top / 448)))
    codes = (c.view(-1, 4, GROUP) / s[..., None]).clamp(-448, 448).reshape(c.shape)
    return codes.to(torch.float8_e4m3fn).view(torch.uint8), s


def visible(row, seqlens, idx):
    """The positions of a row that count, as a list."""
    L = int(seqlens[row])
    if idx is None:
        return list(range(max(L, 0)))
    k = min(idx.shape[1], max(L, 0))
    return [int(t) for t in idx[row, :k] if 0 <= int(t) < L]


def attention_row(q, kv_tokens, scale):
    """One row in 64 bits: q [H, 576], kv_tokens [n, 576] -> out [H, 512], lse [H], and the error
    bounds of a computation with fp32 sums whose weights and result are rounded to bf16."""
    H, n = q.shape[0], kv_tokens.shape[0]
    if n == 0:
        z = torch.zeros(H, LATENT, dtype=torch.float64)
        return z, torch.full((H,), -math.inf, dtype=torch.float64), z, torch.zeros(H, dtype=torch.float64)
    s = scale * (q @ kv_tokens.T)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - lse[:, None])
    c = kv_tokens[:, :LATENT]
    out, size = p @ c, p @ c.abs()
    # a score's fp32 sum of 576 products: at most 576 * 2^-24 of the sum of their magnitudes, in
    # practice the square root's order; 2^-18 leaves a factor of four over 24 * 2^-24
    score = 2.0 ** -18 * (abs(scale) * (q.abs() @ kv_tokens.abs().T)).amax(-1) + 2.0 ** -20
    half = torch.finfo(torch.bfloat16).eps / 2
    bound = half * out.abs() + (half + 2 * score[:, None]) * size * (1 + half)
    return out, lse, bound, score + 2.0 ** -22 * lse.abs()


def numpy_bits(x):
    return x.contiguous().view(torch.uint8).cpu().numpy() if isinstance(x, torch.Tensor) else np.asarray(x)
