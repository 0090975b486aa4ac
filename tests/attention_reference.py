"""Plain 64-bit forms of the attention-layer calls, and the bounds within
which the kernels' results have to lie (numpy-free torch on the CPU)."""
import math

import torch

# a rounding to the type is off by at most this, relative to the value
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
# and by this where the value is below the type's normal range
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def axis_of_pair(rot, sections, interleaved):
    axes = len(sections)
    if not interleaved:
        return [a for a in range(axes) for _ in range(sections[a])]
    return [i % axes if i // axes < sections[i % axes] else 0 for i in range(rot // 2)]


def rotate(x, positions, freqs, sections, pairing, interleaved, inverse=False):
    """x [T][H][D]; positions [axes][T]; returns (y, bound) in 64 bits: the
    rotated x and how far 32-bit arithmetic may be from it before the result
    is rounded.  The reduced turn is narrowed to 32 bits (half a step of at
    most 2^-25 turns, so the angle is off by 2 pi 2^-25 < 2^-22), sine and
    cosine are good to 2^-22, two products and a sum add 2^-23 each."""
    x = x.double()
    rot = 2 * freqs.numel()
    owner = torch.tensor(axis_of_pair(rot, sections, interleaved))
    p = positions.reshape(len(sections), -1).double()
    angle = p[owner].t() * freqs.double()          # [T][rot / 2]
    c, s = torch.cos(angle).unsqueeze(1), torch.sin(angle).unsqueeze(1)
    if inverse:
        s = -s
    if pairing == "halves":
        lo, hi = torch.arange(rot // 2), torch.arange(rot // 2, rot)
    else:
        lo, hi = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    size = (x[..., lo].abs() + x[..., hi].abs())
    # the 64-bit product p f / 2 pi is off by a few 2^-53 of its own size
    far = (angle.abs() * 2.0 ** -50).unsqueeze(1)
    bound[..., lo] = bound[..., hi] = size * (2.0 ** -20 + far)
    return y, bound


def rounded_bound(y, bound, dtype):
    """Bound of y once more rounded to dtype."""
    return bound + (y.abs() + bound) * HALF[dtype] + TINY[dtype]


def attention(q, k, v, scale, causal, window):
    """One sequence: q [n][Hq][D], k, v [kv][Hk][D]; returns (o, weight, spread):
    the result, sum_j p_j |v_j| and the largest sum of |q k| scale, in 64 bits."""
    q, k, v = q.double(), k.double(), v.double()
    n, Hq, D = q.shape
    kv, Hk = k.shape[0], k.shape[1]
    G = Hq // Hk
    o, weight = torch.zeros_like(q), torch.zeros_like(q)
    spread = 0.0
    at = torch.arange(n).unsqueeze(1) + (kv - n)
    key = torch.arange(kv).unsqueeze(0)
    seen = torch.ones(n, kv, dtype=torch.bool)
    if causal:
        seen = key <= at
        if window:
            seen = seen & (key > at - window)
    for h in range(Hq):
        K, V = k[:, h // G], v[:, h // G]
        e = (q[:, h] @ K.t()) * scale
        if n and kv:
            spread = max(spread, float(((q[:, h].abs() @ K.abs().t()) * scale).nan_to_num(
                0, 0, 0).max()))
        for i in range(n):
            w = seen[i]
            if not bool(w.any()):
                continue
            p = torch.softmax(e[i][w], dim=0)
            o[i, h] = p @ V[w]
            weight[i, h] = p @ V[w].abs()
    return o, weight, spread


def attention_bound(o, weight, spread, kv, vmax, D, in_dtype, out_dtype):
    """How far a kernel may be: scores are sums of D exact products in 32 bits
    (relative error D 2^-24 of the sum of their sizes), scaled and shifted by
    one fused operation, and the exponential is good to 2^-21; numerator and
    denominator both carry it, and sums over kv keys in 32 bits.  Two-byte
    results come from probabilities rounded to that type, fp32 ones from
    probabilities of at least 22 bits; an f16 probability below 2^-22 of the
    largest loses up to 2^-33 of it.  The result is rounded once."""
    ds = (D + 4) * 2.0 ** -24 * spread + 2.0 ** -21
    p = HALF[in_dtype] if out_dtype != torch.float32 else 2.0 ** -22
    b = weight * (2 * ds + 2 * (kv + 8) * 2.0 ** -24 + p)
    if in_dtype == torch.float16:
        b = b + kv * 2.0 ** -33 * vmax
    return rounded_bound(o, b, out_dtype)
