"""Plain 64-bit forms of the calls around per-head norms and 4-bit caches, and
the bounds within which the kernels' results have to lie (torch on the CPU)."""
import torch

import attention_reference as ref

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
EXPONENTS = {torch.bfloat16: (-100, 125), torch.float16: (-23, 13)}


def values(codes, scales):
    """What codes [..., D / 2] and scales [..., D / 32] (uint8) stand for."""
    c = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    x = torch.where(c >= 8, -1.0, 1.0).double() * GRID[c % 8]
    s = torch.pow(torch.tensor(2.0, dtype=torch.float64), scales.double() - 127)
    s = torch.where(scales == 255, torch.nan, s)
    return x * s.repeat_interleave(32, dim=-1)


def quantise(x, dtype):
    """What a cache of this dtype holds of x [..., D]: (values, scale bytes).  The
    scale by trying exponents from the least, the code by trying all."""
    lo, hi = EXPONENTS[dtype]
    g = x.double().unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    fine = torch.isfinite(g).all(-1, keepdim=True)
    e = torch.full_like(top, lo)
    for n in range(lo, hi):
        e = torch.where(top > 7.0 * 2.0 ** n, n + 1.0, e)
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), e)
    a = (g.abs() / unit).clamp_max(6.0)
    # even codes first: argmin takes the first of equals
    order = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7])
    best = GRID[order][torch.argmin((a.unsqueeze(-1) - GRID[order]).abs(), dim=-1)]
    y = torch.where(fine, torch.copysign(best * unit, g), torch.nan)
    return y.flatten(-2), torch.where(fine, e + 127, 255.0).squeeze(-1).to(torch.uint8)


def encode(y, byte):
    """Codes [..., D / 2] of values that a cache with these scales holds."""
    unit = torch.pow(torch.tensor(2.0, dtype=torch.float64), byte.double() - 127)
    a = (y.abs().unflatten(-1, (-1, 32)) / unit.unsqueeze(-1)).flatten(-2)
    code = (a.unsqueeze(-1) >= GRID[1:]).sum(-1) + 8 * torch.signbit(y)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def attention(q, k, v, scale, causal, window, sinks):
    """attention_reference.attention with the first `sinks` keys visible as well."""
    q, k, v = q.double(), k.double(), v.double()
    n, Hq, D = q.shape
    kv, G = k.shape[0], Hq // k.shape[1]
    o, weight, spread = torch.zeros_like(q), torch.zeros_like(q), 0.0
    for i in range(n):
        at = kv - n + i
        seen = [j for j in range(kv) if not causal or (
            j <= at and (not window or j > at - window or j < sinks))]
        if not seen:
            continue
        for h in range(Hq):
            K, V = k[seen, h // G], v[seen, h // G]
            e = (K @ q[i, h]) * scale
            spread = max(spread, float(((K.abs() @ q[i, h].abs()) * scale).nan_to_num(0, 0, 0).max()))
            p = torch.softmax(e, dim=0)
            o[i, h], weight[i, h] = p @ V, p @ V.abs()
    return o, weight, spread


def root(x, eps):
    """r of each head."""
    return (x.double().square().mean(-1, keepdim=True) + eps).rsqrt()


def norm_rope(x, w, eps, positions=None, freqs=None, sections=None, pairing="halves",
              interleaved=False, inverse=False):
    """(y, bound) in 64 bits.  In 32 bits r is off by 2^-25 (its square was
    narrowed) and two roundings, x r w by two more: below 2^-21 of the value in
    all; the rotation's own bound is attention_reference.rotate's.  Below fp32's
    normal range each rounding is off by up to 2^-150 instead: x times the power
    of two in r, that times the rest of r (below 1.5, so by 1.5 2^-150 + 2^-150
    then) and times w: (2.5 |w| + 1) 2^-150 in all."""
    z = x.double() * root(x, eps) * w.double()
    least = (2.5 * w.double().abs() + 1) * 2.0 ** -150
    if freqs is None:
        return z, z.abs() * 2.0 ** -21 + least
    y, bound = ref.rotate(z, positions, freqs, sections, pairing, interleaved, inverse)
    # each result takes two of z at most: their sizes sum to no more than this
    size, _ = ref.rotate(z.abs(), positions * 0, freqs, sections, pairing, interleaved)
    rot = 2 * freqs.numel()
    pair = torch.zeros_like(z)
    if pairing == "halves":
        lo, hi = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    else:
        lo, hi = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    pair[..., lo] = size[..., hi]
    pair[..., hi] = size[..., lo]
    # two products and a sum below the normal range: 3 2^-150 more
    return y, bound + (size + pair) * 2.0 ** -21 + 2 * least.max() + 3 * 2.0 ** -150


def norm_rope_grad(g, x, w, eps, positions=None, freqs=None, sections=None, pairing="halves",
                   interleaved=False, inverse=False):
    """(dx, its bound, dw, its bound) in 64 bits.  u is off by the rotation's
    bound, n = x r by 3 2^-24 of itself, products and their mean by a few 2^-24;
    dw is summed over a thread's heads and a workgroup's 256 threads in 32 bits."""
    T, H, D = x.shape
    u, eu = g.double(), torch.zeros_like(g, dtype=torch.float64)
    if freqs is not None:
        u, eu = ref.rotate(u, positions, freqs, sections, pairing, interleaved, not inverse)
    r, w = root(x, eps), w.double()
    n = x.double() * r
    along = (w * u * n).sum(-1, keepdim=True) / D
    off = (w.abs() * (eu + u.abs() * 2.0 ** -21) * n.abs()).sum(-1, keepdim=True) / D
    dx = r * (w * u - n * along)
    bx = r * (w.abs() * eu + n.abs() * off + 2.0 ** -21 * ((w * u).abs() + (n * along).abs()))
    dw = (u * n).sum((0, 1))
    count = (9 + H) * (T // 1024 + 1) + 256
    bw = ((eu + u.abs() * (2.0 ** -21 + count * 2.0 ** -24)) * n.abs()).sum((0, 1))
    return dx, bx, dw, bw + dw.abs() * 2.0 ** -24
