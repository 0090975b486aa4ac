"""Timed cases of the attention-layer operators around a cache held in 4 bits:
norms of queries and keys with the rotation in the same pass (and their
gradient), the append that quantises on the way, reading such a cache back,
attention over it, and attention in a sliding window whose first few tokens
stay visible.

The cache holds e2m1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign), and a power
of two for each 32 neighbours of a head.  Head shapes are those of the tested
27B model (24 query heads, 4 key heads, 256 wide, 64 of them rotated over time,
height and width) next to generic ones.

``own`` False computes each operator from elementary torch operations in 32
bits (64 for angles, for sums over all tokens and for what is quantised);
``own`` True calls the library.
"""
import math
import random

import torch

own = False

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
_DT = {"f32": F32, "bf16": BF16, "f16": F16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_BASE = 1.0e6  # frequency base of the rotation
_EPS = 1.0e-6
_GROUP = 32    # neighbours that share a scale


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _norm(name, way, T, H, D, rot, sections, pairing, interleaved, din, dout, far):
    return {"name": name, "op": "norm", "way": way, "T": T, "H": H, "D": D, "rot": rot,
            "sections": sections, "pairing": pairing, "interleaved": interleaved, "din": din,
            "dout": dout, "far": far}


def _append(name, bits, norm, T, B, pad, Hk, G, D, rot, sections, pairing, interleaved, page, din,
            dtype, far):
    return {"name": name, "op": "append", "bits": bits, "norm": norm, "T": T, "B": B, "pad": pad,
            "Hk": Hk, "G": G, "D": D, "rot": rot, "sections": sections, "pairing": pairing,
            "interleaved": interleaved, "page": page, "din": din, "dtype": dtype, "far": far}


def _read(name, T, Hk, D, page, dtype, dout):
    return {"name": name, "op": "read", "T": T, "Hk": Hk, "D": D, "page": page, "dtype": dtype,
            "dout": dout}


def _attention(name, bits, B, q_min, q_max, past_min, past_max, Hk, G, D, page, dtype, dout, causal,
               window, sinks):
    return {"name": name, "op": "attention", "bits": bits, "B": B, "q_min": q_min, "q_max": q_max,
            "past_min": past_min, "past_max": past_max, "Hk": Hk, "G": G, "D": D, "page": page,
            "dtype": dtype, "dout": dout, "causal": causal, "window": window, "sinks": sinks}


def listed():
    return [
        # the queries of one decoded token, straight from the fp32 projection
        _norm("norm one token", "forward", 1, 24, 256, 64, "11,11,10", "halves", True, "f32", "bf16",
              5000),
        # the queries of a long prompt
        _norm("norm prompt", "forward", 8190, 24, 256, 64, "11,11,10", "halves", True, "bf16", "bf16",
              0),
        # training: gradient of the queries and of the norm's weight
        _norm("norm gradient", "gradient", 8190, 24, 256, 64, "11,11,10", "halves", True, "bf16",
              "bf16", 0),
        # a batch of users decoding, the batch padded to a fixed size
        _append("append decode batch", 4, True, 96, 91, 5, 8, 4, 128, 128, "64", "halves", False, 16,
                "f16", "f16", 20000),
        # three prompts entering the cache together
        _append("append prompts", 4, True, 4001, 3, 0, 4, 6, 256, 64, "11,11,10", "halves", True, 64,
                "f32", "bf16", 0),
        # a short prefix that another sequence shares, widened for its copy
        _read("read prefix", 333, 4, 256, 16, "bf16", "bf16"),
        # a long document's keys and values, handed to a 16-bit cache
        _read("read document", 50000, 4, 256, 64, "bf16", "bf16"),
        # one user early in a conversation; fp32 out for the rotation of the output projection
        _attention("attend one token", 4, 1, 1, 1, 700, 700, 4, 6, 256, 16, "bf16", "f32", True, 0, 0),
        # a batch of users decoding at their own lengths
        _attention("attend decode batch", 4, 64, 1, 1, 200, 8000, 4, 6, 256, 64, "bf16", "bf16", True,
                   0, 0),
        # a chunk of a long prompt after the part already in the cache
        _attention("attend prompt chunk", 4, 1, 2048, 2048, 6144, 6144, 4, 6, 256, 64, "bf16", "bf16",
                   True, 0, 0),
        # streams that never end: a window and the first tokens, 16-bit cache
        _attention("attend streams", 16, 48, 1, 1, 2000, 30000, 8, 4, 128, 32, "f16", "f16", True,
                   1024, 4),
        # whole prompts of ragged lengths of a model with such layers, 16-bit cache
        _attention("attend prompts in a window", 16, 3, 500, 6000, 0, 0, 4, 6, 256, 64, "bf16", "bf16",
                   True, 1024, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rotation(rng, D, partial):
    """rot, sections, interleaved: up to four axes over rot / 2 pairs."""
    rot = D if not partial else rng.choice([D // 4 // 2 * 2, D // 2 // 2 * 2, D])
    half = rot // 2
    axes = rng.choice([1, 1, 2, 3, 3, 4])
    base, extra = divmod(half, axes)
    sec = [base + (1 if a < extra else 0) for a in range(axes)]
    interleaved = axes > 1 and rng.random() < 0.5
    if axes > 1 and not interleaved and rng.random() < 0.5:
        k = rng.randrange(0, sec[1])
        sec[0], sec[1] = sec[0] + k, sec[1] - k
    return rot, ",".join(str(s) for s in sec), interleaved


def draw(rng):
    kind = rng.choice(["norm", "append", "read", "attention", "attention", "attention"])
    if kind == "norm":
        D = rng.choice([64, 72, 80, 96, 128, 128, 256])
        H = rng.choice([1, 4, 8, 16, 24, 32])
        T = _log(rng, 1, min(8000, 48_000_000 // (H * D)))
        rot, sec, inter = _draw_rotation(rng, D, rng.random() < 0.5)
        if rng.random() < 0.15:
            rot, sec, inter = 0, "", False
        c = _norm("", rng.choice(["forward", "gradient"]), T, H, D, rot, sec,
                  rng.choice(["halves", "halves", "adjacent"]), inter,
                  rng.choice(["f32", "bf16", "f16"]), None, rng.choice([0, 0, 10000, 500000]))
        c["dout"] = rng.choice([c["din"], {"f32": "bf16"}.get(c["din"], c["din"])])
        if c["way"] == "gradient":
            c["dout"] = c["din"]
    elif kind == "append":
        D = rng.choice([64, 96, 128, 256])
        Hk, G = rng.choice([(1, 8), (2, 7), (4, 6), (4, 6), (8, 4), (8, 1), (4, 0)])
        T = _log(rng, 1, min(4000, 30_000_000 // ((2 + G) * Hk * D)))
        B = rng.choice([1, max(1, T // 100), min(T, 64)])
        rot, sec, inter = _draw_rotation(rng, D, rng.random() < 0.5)
        if rng.random() < 0.15:
            rot, sec, inter = 0, "", False
        pad = 0 if T < 4 else rng.choice([0, 0, min(3, T - B)])
        dt = rng.choice(["bf16", "f16"])
        bits = rng.choice([4, 4, 4, 16])
        c = _append("", bits, bits == 16 or rng.random() < 0.7, T, B, pad, Hk, G, D, rot, sec,
                    rng.choice(["halves", "adjacent"]), inter, rng.choice([1, 8, 16, 32, 64, 128]),
                    rng.choice(["f32", dt]), dt, rng.choice([0, 10000, 500000]))
    elif kind == "read":
        D = rng.choice([32, 64, 96, 128, 256])
        Hk = rng.choice([1, 2, 4, 8])
        T = _log(rng, 1, min(50000, 50_000_000 // (Hk * D)))
        dt = rng.choice(["bf16", "f16"])
        c = _read("", T, Hk, D, rng.choice([1, 8, 16, 32, 64, 128]), dt, rng.choice([dt, dt, "f32"]))
    else:
        D = rng.choice([64, 128, 256])
        Hk, G = rng.choice([(1, 8), (2, 7), (4, 6), (4, 6), (8, 4), (8, 1), (2, 16)])
        shape = rng.choice(["decode", "decode", "drafts", "chunk", "prompt"])
        q_max = {"decode": 1, "drafts": rng.randint(2, 8), "chunk": _log(rng, 9, 2000),
                 "prompt": _log(rng, 2, 4000)}[shape]
        q_min = q_max if rng.random() < 0.5 else rng.randint(1, q_max)
        past = 0 if shape == "prompt" else _log(rng, 1, 60000 if shape == "decode" else 8000)
        B = _log(rng, 1, 64)
        bits = rng.choice([4, 4, 16])
        window = rng.randint(1, 4000) if bits == 16 else rng.choice([0, 0, rng.randint(1, 4000)])
        sinks = rng.choice([1, 4, 16, _log(rng, 1, 300)]) if window and (
            bits == 16 or rng.random() < 0.7) else 0
        causal = True if window else rng.random() < 0.85
        dt = rng.choice(["bf16", "bf16", "f16"])
        c = _attention("", bits, B, q_min, q_max, rng.randint(0, past), past, Hk, G, D,
                       rng.choice([1, 8, 16, 32, 64, 128, 256]), dt,
                       rng.choice([dt, dt, "f32"]), causal, window, sinks)
        # no more than the largest listed cases, in products, in bytes and in pairs of the plain form
        cost = lambda: (work(c)["flops"] > 3.5e11 or work(c)["bytes"] > 2.9e8
                        or _lens(c)[2] * Hk * G > 1.0e9)
        while c["B"] > 1 and cost():
            c["B"] = c["B"] // 2
        while cost():
            c["q_max"] = max(1, c["q_max"] // 2)
            c["q_min"] = min(c["q_min"], c["q_max"])
            c["past_max"] //= 2
            c["past_min"] = min(c["past_min"], c["past_max"])
    while c["op"] != "attention" and work(c)["bytes"] > 2.9e8:
        c["T"] //= 2
    del c["name"]
    return c


def _lens(case):
    """New tokens and cached tokens of every sequence, and all pairs of them: a
    function of the case alone, so that its work is known without its inputs."""
    rng = random.Random(case["B"] * 1000003 + case["q_max"] * 1009 + case["past_max"])
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["B"])]
    past = [rng.randint(case["past_min"], case["past_max"]) for _ in range(case["B"])]
    q[0] = case["q_max"]
    past[0] = case["past_max"]
    return q, past, sum(n * (n + p) for n, p in zip(q, past))


def _seen(case, n, past):
    """(query, key) pairs of one sequence that the mask leaves, and its keys that are read."""
    kv = n + past
    if not case["causal"]:
        return n * kv, kv
    w, s = case["window"] or kv, case["sinks"]
    pairs = keys = 0
    for i in range(n):                       # row i stands at past + i
        end = past + i + 1
        lo = max(0, end - w)
        pairs += end - lo + min(s, lo)
    first = max(0, past + 1 - w)             # of the first row; later rows see later keys
    keys = kv - first + min(s, first)
    return pairs, keys


def work(case):
    if case["op"] == "norm":
        n = case["T"] * case["H"] * case["D"]
        axes = len(_sections(case))
        small = 4 * axes * case["T"] + 4 * case["rot"] + 4 * case["D"]
        if case["way"] == "forward":
            return {"bytes": n * (_SIZE[case["din"]] + _SIZE[case["dout"]]) + small,
                    "flops": 4 * n + 3 * case["T"] * case["H"] * case["rot"]}
        return {"bytes": 3 * n * _SIZE[case["din"]] + small + 4 * case["D"],
                "flops": 10 * n + 3 * case["T"] * case["H"] * case["rot"]}
    if case["op"] == "append":
        T, live = case["T"], case["T"] - case["pad"]
        kv, q = 2 * case["Hk"] * case["D"], case["Hk"] * case["G"] * case["D"]
        axes = len(_sections(case))
        held = kv * (0.5 + 1 / _GROUP if case["bits"] == 4 else 2)
        # the cache's values, which this case returns, are not part of what an append has to move
        return {"bytes": live * (kv * _SIZE[case["din"]] + held)
                + T * q * (_SIZE[case["din"]] + _SIZE[case["dtype"]]) + T * (8 + 4 * axes)
                + 4 * case["rot"] + 8 * case["D"],
                "flops": 4 * T * (kv + q) + 3 * T * case["Hk"] * (1 + case["G"]) * case["rot"]}
    if case["op"] == "read":
        n = 2 * case["T"] * case["Hk"] * case["D"]
        return {"bytes": n * (0.5 + 1 / _GROUP + _SIZE[case["dout"]]) + 8 * case["T"], "flops": n}
    qs, pasts, _ = _lens(case)
    Hq = case["Hk"] * case["G"]
    pairs = keys = pages = 0
    for n, p in zip(qs, pasts):
        a, b = _seen(case, n, p)
        pairs, keys, pages = pairs + a, keys + b, pages + -(-b // case["page"])
    rows = sum(qs) * Hq
    held = 1 + 2 / _GROUP if case["bits"] == 4 else 4   # bytes of a key's and a value's element
    return {"bytes": rows * case["D"] * (2 + _SIZE[case["dout"]]) + keys * case["Hk"] * case["D"] * held
            + 4 * pages + 4 * (2 * case["B"] + 1), "flops": 4 * pairs * Hq * case["D"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _sections(case):
    return [int(s) for s in case["sections"].split(",")] if case["sections"] else []


def _positions(case, T, g):
    """[axes][T] int32: text positions, then (for several axes) the rows and columns of an image."""
    axes = len(_sections(case))
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    start = torch.randint(0, 64, (axes, 1), device="cuda", generator=g, dtype=torch.int32)
    if axes == 1:
        return (t.unsqueeze(0) + start + case["far"]).contiguous()
    side = max(1, math.isqrt(T))
    rows = [t, t // side, t % side, t // (side * side)][:axes]
    return (torch.stack(rows) + start + case["far"]).contiguous()


def _freqs(rot):
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    return torch.pow(torch.tensor(_BASE, dtype=torch.float64, device="cuda"), -2.0 * i / rot)


def _weight(D, g):
    return 1.0 + 0.2 * torch.randn(D, device="cuda", generator=g)


def _exponents(dtype):
    """Least and largest exponent of a scale: what the type that the values are read in holds."""
    return (-100, 125) if dtype == "bf16" else (-23, 13)


def _quantise(x, dtype):
    """Codes [..., D / 2] (two of them in a byte, the first in its low half) and
    scales [..., D / 32] (exponent + 127; 255 for a group that is not finite)."""
    shape = x.shape
    x = x.unflatten(-1, (-1, _GROUP))
    top = x.abs().amax(dim=-1, keepdim=True)
    fine = torch.isfinite(top)
    m, e = torch.frexp(torch.where(fine, top, torch.ones_like(top)))  # top = m 2^e, m in [0.5, 1)
    lo, hi = _exponents(dtype)
    e = (e - 3 + (m > 0.875).to(e.dtype)).clamp(lo, hi)
    e = torch.where(top > 0, e, torch.full_like(e, lo))
    a = torch.ldexp(x.abs(), -e)
    code = sum((a >= b if even else a > b).to(torch.uint8) for b, even in
               ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                (5.0, False)))
    code = code + 8 * torch.signbit(x).to(torch.uint8)
    code = torch.where(fine, code, torch.zeros_like(code)).reshape(shape)
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8).squeeze(-1)
    return code[..., 0::2] + 16 * code[..., 1::2], scale


def _values(codes, scales):
    """What codes and scales stand for, in 32 bits."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    code = torch.stack([codes & 15, codes >> 4], dim=-1).flatten(-2).long()
    x = table[code & 7] * (1.0 - 2.0 * (code >> 3).float())
    s = torch.exp2(scales.float() - 127.0)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return (x.unflatten(-1, (-1, _GROUP)) * s.unsqueeze(-1)).flatten(-2)


def _cache(case, pages, g):
    """Keys and values of earlier tokens, as the cache holds them."""
    shape = (pages, case["Hk"], case["page"], case["D"])
    dt = _DT[case["dtype"]]
    if case.get("bits", 4) == 16:
        return tuple(torch.randn(shape, device="cuda", generator=g).to(dt) for _ in range(2))
    held = []
    for _ in range(2):
        codes = torch.empty((*shape[:3], shape[3] // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((*shape[:3], shape[3] // _GROUP), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 25) // (shape[1] * shape[2] * shape[3]))
        for p in range(0, pages, step):
            part = torch.randn((min(step, pages - p), *shape[1:]), device="cuda", generator=g)
            codes[p:p + step], scales[p:p + step] = _quantise(part, case["dtype"])
        held += [codes, scales]
    return tuple(held)


def _inputs(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, H, D = case["T"], case["H"], case["D"]
        s["x"] = (3.0 * torch.randn(T, H, D, device="cuda", generator=g)).to(_DT[case["din"]])
        s["w"] = _weight(D, g)
        if case["way"] == "gradient":
            s["g"] = torch.randn(T, H, D, device="cuda", generator=g).to(_DT[case["din"]])
        if case["rot"]:
            s["positions"] = _positions(case, T, g)
            s["freqs"] = _freqs(case["rot"])
    elif case["op"] == "append":
        T, B, Hk, G, D, page = (case[k] for k in ("T", "B", "Hk", "G", "D", "page"))
        # the stacked projection's output: queries, keys and values of a token side by side
        qkv = torch.randn(T, (G + 2) * Hk * D, device="cuda", generator=g).to(_DT[case["din"]])
        s["q"] = qkv[:, :G * Hk * D].unflatten(1, (G * Hk, D)) if G else None
        s["k"] = qkv[:, G * Hk * D:(G + 1) * Hk * D].unflatten(1, (Hk, D))
        s["v"] = qkv[:, (G + 1) * Hk * D:].unflatten(1, (Hk, D))
        live = T - case["pad"]
        each = -(-live // B)                  # new tokens of a sequence
        per = -(-each // page) + 1            # pages it may touch
        pages = B * per + 3
        order = torch.randperm(pages, device="cuda", generator=g)[:B * per].view(B, per)
        first = torch.randint(0, page, (B,), device="cuda", generator=g)
        t = torch.arange(live, device="cuda")
        b, i = t // each, t % each
        at = first[b] + i
        slots = order[b, at // page] * page + at % page
        s["slots"] = torch.full((T,), -1, dtype=torch.int64, device="cuda")
        s["slots"][:live] = slots
        s["held"] = _cache(case, pages, g)
        s["all"] = torch.arange(pages * page, device="cuda")
        if case["norm"]:
            s["qw"], s["kw"] = _weight(D, g), _weight(D, g)
        if case["rot"]:
            s["positions"] = _positions(case, T, g)
            s["freqs"] = _freqs(case["rot"])
    elif case["op"] == "read":
        T, page = case["T"], case["page"]
        pages = -(-T // page) + 2
        s["held"] = _cache(case, pages, g)
        order = torch.randperm(pages, device="cuda", generator=g)
        t = torch.arange(T, device="cuda")
        s["slots"] = order[t // page] * page + t % page
    else:
        Hk, G, D, page = (case[k] for k in ("Hk", "G", "D", "page"))
        qs, pasts, _ = _lens(case)
        need = [-(-(n + p) // page) for n, p in zip(qs, pasts)]
        pages = sum(need) + 5
        order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
        table = torch.full((case["B"], max(need) + 1), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, c in enumerate(need):
            table[b, :c] = order[at:at + c]
            at += c
        s["table"] = table
        # normalised heads, somewhat peaked scores
        s["q"] = (1.5 * torch.randn(sum(qs), Hk * G, D, device="cuda", generator=g)).to(
            _DT[case["dtype"]])
        s["held"] = _cache(case, pages, g)
        cu = [0]
        for n in qs:
            cu.append(cu[-1] + n)
        s["cu_host"], s["kv_host"] = cu, [n + p for n, p in zip(qs, pasts)]
        s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        s["kv"] = torch.tensor(s["kv_host"], dtype=torch.int32, device="cuda")
        s["max_q"], s["max_kv"] = max(qs), max(s["kv_host"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from gemm_hadamard_rotated_amd import pq1
        if case.get("rot"):
            s["rope"] = pq1.Rope(case["rot"], _sections(case), freqs=s["freqs"],
                                 pairing=case["pairing"], interleaved=case["interleaved"])
        if case.get("norm"):
            s["norm"] = pq1.HeadNorm(s["kw"], s["qw"] if s["q"] is not None else None, eps=_EPS)
        if "held" in s:
            s["cache"] = pq1.KVCache(*s["held"]) if case.get("bits", 4) == 16 else \
                pq1.KV4Cache(*s["held"], dtype=_DT[case["dtype"]])
    elif case.get("rot"):
        s["axis"] = torch.tensor(_axis_of_pair(case), device="cuda")
    return s


def _axis_of_pair(case):
    """Position axis of every rotated pair.  In order: the first section's
    pairs, then the second's; interleaved: axis i % axes while that axis's
    section lasts, the first axis otherwise."""
    sec = _sections(case)
    if not case["interleaved"]:
        return [a for a, n in enumerate(sec) for _ in range(n)]
    out = []
    for i in range(case["rot"] // 2):
        a = i % len(sec)
        out.append(a if i // len(sec) < sec[a] else 0)
    return out


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from gemm_hadamard_rotated_amd import pq1
    case = s["case"]
    if case["op"] == "norm":
        if case["way"] == "forward":
            return pq1.pq1_norm_rope(s["x"], s["w"], s.get("positions"), s.get("rope"), eps=_EPS,
                                     out_dtype=_DT[case["dout"]])
        return pq1.pq1_norm_rope_grad(s["g"], s["x"], s["w"], s.get("positions"), s.get("rope"),
                                      eps=_EPS)
    if case["op"] == "append":
        if case["bits"] == 16:
            q_out = pq1.pq1_kv_append(s["cache"], s["k"], s["v"], s["slots"],
                                      positions=s.get("positions"), rope=s.get("rope"), q=s["q"],
                                      norm=s["norm"])
            out = s["held"]
        else:
            q_out = pq1.pq1_kv4_append(s["cache"], s["k"], s["v"], s["slots"],
                                       positions=s.get("positions"), rope=s.get("rope"), q=s["q"],
                                       norm=s.get("norm"))
            out = tuple(pq1.pq1_kv4_read(s["cache"], s["all"]))
        return out if q_out is None else out + (q_out,)
    if case["op"] == "read":
        return tuple(pq1.pq1_kv4_read(s["cache"], s["slots"], out_dtype=_DT[case["dout"]]))
    attend = pq1.pq1_paged_attention if case["bits"] == 16 else pq1.pq1_kv4_attention
    return attend(s["q"], s["cache"], s["table"], s["cu"], s["kv"], max_q=s["max_q"],
                  max_kv=s["max_kv"], causal=case["causal"], window=case["window"],
                  sinks=case["sinks"], out_dtype=_DT[case["dout"]])


def _turn_plain(x, s, inverse=False):
    """x [T][H][D] rotated in x's own bits; angles in 64 bits, reduced before they are narrowed."""
    case = s["case"]
    rot = case["rot"]
    if not rot:
        return x
    angle = s["positions"].double()[s["axis"]].t() * s["freqs"]
    angle = torch.remainder(angle, 2.0 * math.pi).to(x.dtype).unsqueeze(1)
    c, n = torch.cos(angle), torch.sin(angle)
    if inverse:
        n = -n
    y = x.clone()
    if case["pairing"] == "halves":
        lo, hi = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        lo, hi = slice(0, rot, 2), slice(1, rot, 2)
    y[..., lo] = x[..., lo] * c - x[..., hi] * n
    y[..., hi] = x[..., hi] * c + x[..., lo] * n
    return y


def _norm_plain(x, w):
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + _EPS) * w


def _rows(x):
    """[pages][heads][page][n] as [slots][heads][n]."""
    return x.transpose(1, 2).flatten(0, 1)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        x, w = s["x"].float(), s["w"]
        if case["way"] == "forward":
            return _turn_plain(_norm_plain(x, w), s).to(_DT[case["dout"]])
        u = _turn_plain(s["g"].float(), s, inverse=True)
        r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + _EPS)
        dw = (u * x * r).sum(dim=(0, 1), dtype=torch.float64).float()
        uw = u * w
        dx = r * uw - x * (r * r * r * (uw * x).mean(dim=-1, keepdim=True))
        return dx.to(s["x"].dtype), dw
    if case["op"] == "append":
        dt, page = _DT[case["dtype"]], case["page"]
        wide = F32 if case["bits"] == 16 else torch.float64   # next to a border 32 bits are too few
        k, v = s["k"].to(wide), s["v"].to(wide)
        if case["norm"]:
            k = _norm_plain(k, s["kw"].to(wide))
        k = _turn_plain(k, s)
        live = torch.nonzero(s["slots"] >= 0).squeeze(1)
        at = s["slots"][live]
        new = (k[live].to(dt), v[live].to(dt)) if case["bits"] == 16 else \
            (*_quantise(k[live], case["dtype"]), *_quantise(v[live], case["dtype"]))
        for held, x in zip(s["held"], new):
            held[at // page, :, at % page] = x
        out = s["held"] if case["bits"] == 16 else tuple(
            _rows(_values(*s["held"][i:i + 2])).to(dt) for i in (0, 2))
        if s["q"] is None:
            return out
        q = s["q"].float()
        if case["norm"]:
            q = _norm_plain(q, s["qw"])
        return out + (_turn_plain(q, s).to(dt),)
    if case["op"] == "read":
        page, at = case["page"], s["slots"]
        where, off = at // page, at % page
        return tuple(_values(s["held"][i][where, :, off], s["held"][i + 1][where, :, off]).to(
            _DT[case["dout"]]) for i in (0, 2))
    Hk, G, D, page = (case[k] for k in ("Hk", "G", "D", "page"))
    out = torch.zeros(s["q"].shape, dtype=_DT[case["dout"]], device="cuda")
    for b in range(case["B"]):
        q0, q1, kv = s["cu_host"][b], s["cu_host"][b + 1], s["kv_host"][b]
        n = q1 - q0
        key = torch.arange(kv, device="cuda")
        where, off = s["table"][b, key // page].long(), key % page
        rows = [x[where, :, off] for x in s["held"]]
        K, V = (x.float() for x in rows) if case["bits"] == 16 else \
            (_values(*rows[:2]), _values(*rows[2:]))
        K = K.permute(1, 2, 0).contiguous()   # [Hk][D][kv]
        V = V.permute(1, 0, 2).contiguous()   # [Hk][kv][D]
        q = s["q"][q0:q1].float().view(n, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * n, D)
        score = torch.matmul(q, K).view(Hk, G, n, kv) * (1.0 / math.sqrt(D))
        if case["causal"]:
            at = torch.arange(n, device="cuda").unsqueeze(1) + (kv - n)
            hidden = key > at
            if case["window"]:
                hidden = hidden | ((key <= at - case["window"]) & (key >= case["sinks"]))
            score = score.masked_fill(hidden, -math.inf)
        top = score.amax(dim=-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(score - top)
        total = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.view(Hk, G * n, kv), V).view(Hk, G, n, D)
        o = torch.where(total > 0, o / total, torch.zeros_like(o))
        out[q0:q1] = o.permute(2, 0, 1, 3).reshape(n, Hk * G, D).to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# 64-bit values
# ---------------------------------------------------------------------------
def _turn_exact(x, positions, case, inverse=False):
    """Each pair as a complex number times exp(i pos f)."""
    rot, half = case["rot"], case["rot"] // 2
    if not rot:
        return x
    sec = _sections(case)
    owner = torch.zeros(half, dtype=torch.int64)
    if case["interleaved"]:
        for a in range(1, len(sec)):
            owner[a:a + len(sec) * sec[a]:len(sec)] = a
    else:
        owner = torch.repeat_interleave(torch.arange(len(sec)), torch.tensor(sec))
    f = torch.tensor([_BASE ** (-2.0 * i / rot) for i in range(half)], dtype=torch.float64)
    turn = positions.cpu().double()[owner].t() * f
    z = torch.polar(torch.ones_like(turn), -turn if inverse else turn).to(x.device).unsqueeze(1)
    head = x[..., :rot]
    if case["pairing"] == "halves":
        w = torch.complex(head[..., :half], head[..., half:]) * z
        turned = torch.cat([w.real, w.imag], dim=-1)
    else:
        w = torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * z
        turned = torch.view_as_real(w).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _unit(x, w):
    """x over the root of its mean square, times w."""
    return w.double() * x / (torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / x.shape[-1]
                             + _EPS).sqrt()


def _held_exact(x, dtype):
    """The value that a 4-bit cache holds for each of x: the nearest of 15 multiples of the
    least power of two that leaves the group's largest at 7 or below (even codes win ties)."""
    grid = torch.tensor([0.0, 1.0, 2.0, 4.0, 0.5, 1.5, 3.0, 6.0], dtype=torch.float64, device=x.device)
    y = torch.empty_like(x)
    lo, hi = _exponents(dtype)
    for g in range(0, x.shape[-1], _GROUP):
        part = x[..., g:g + _GROUP]
        top = part.abs().amax(-1, keepdim=True).clamp_min(2.0 ** -1000)
        unit = torch.pow(2.0, torch.ceil(torch.log2(top / 7.0)).clamp(lo, hi).double())
        unit = torch.where((top > 7.0 * unit) & (unit < 2.0 ** hi), 2.0 * unit, unit)
        unit = torch.where((top <= 3.5 * unit) & (unit > 2.0 ** lo), 0.5 * unit, unit)
        a = (part.abs() / unit).clamp_max(6.0)
        best = grid[torch.argmin((a.unsqueeze(-1) - grid).abs(), dim=-1)]
        y[..., g:g + _GROUP] = torch.copysign(best * unit, part)
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm":
        x, w, pos = s["x"].double(), s["w"].double(), s.get("positions")
        if case["way"] == "forward":
            return _turn_exact(_unit(x, w), pos, case)
        u = _turn_exact(s["g"].double(), pos, case, inverse=True)
        size = (torch.linalg.vector_norm(x, dim=-1, keepdim=True).square() / case["D"] + _EPS).sqrt()
        unit = x / size
        dw = (u * unit).sum(dim=(0, 1))
        along = (u * w * unit).sum(-1, keepdim=True) / case["D"]
        return (u * w - along * unit) / size, dw
    if case["op"] == "append":
        k, v, pos = s["k"].double(), s["v"].double(), s.get("positions")
        if case["norm"]:
            k = _unit(k, s["kw"])
        k = _turn_exact(k, pos, case)
        used = s["slots"] >= 0
        out = []
        for i, new in enumerate((k, v)):
            if case["bits"] == 16:
                flat = _rows(s["held"][i].double()).contiguous()
                flat.index_copy_(0, s["slots"][used], new[used])
                out.append(flat.view(-1, case["page"], case["Hk"], case["D"]).transpose(1, 2)
                           .contiguous())
            else:
                flat = _rows(_values(*s["held"][2 * i:2 * i + 2])).double().contiguous()
                flat.index_copy_(0, s["slots"][used], _held_exact(new[used], case["dtype"]))
                out.append(flat)
        if s["q"] is None:
            return tuple(out)
        q = s["q"].double()
        return (*out, _turn_exact(_unit(q, s["qw"]) if case["norm"] else q, pos, case))
    if case["op"] == "read":
        out = []
        for i in (0, 2):
            c = _rows(s["held"][i])[s["slots"]].to(torch.int16)
            e = _rows(s["held"][i + 1])[s["slots"]].double() - 127.0
            c = torch.stack([c % 16, c // 16], dim=-1).flatten(-2)
            a, m = (c % 8) // 2, c % 2                   # exponent and mantissa bit of e2m1
            x = torch.where(a > 0, (1.0 + 0.5 * m) * torch.pow(2.0, a.double() - 1.0), 0.5 * m.double())
            x = torch.where(c >= 8, -x, x) * torch.pow(2.0, e).repeat_interleave(_GROUP, dim=-1)
            out.append(x)
        return tuple(out)
    Hk, G, D = case["Hk"], case["G"], case["D"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        q0, q1, kv = s["cu_host"][b], s["cu_host"][b + 1], s["kv_host"][b]
        n, used = q1 - q0, -(-kv // case["page"])
        rows = s["table"][b, :used].long()
        seen = torch.ones(n, kv, dtype=torch.bool, device="cuda")
        if case["causal"]:
            seen = seen.tril(kv - n)
            if case["window"]:
                near = seen.triu(kv - n - case["window"] + 1)
                near[:, :case["sinks"]] = seen[:, :case["sinks"]]
                seen = near
        for h in range(Hk):
            part = [x[rows, h] for x in s["held"]]
            if case["bits"] == 4:
                part = [_values(*part[:2]), _values(*part[2:])]
            K, V = (x.reshape(-1, D)[:kv].double() for x in part)
            for j in range(h * G, (h + 1) * G):
                e = (s["q"][q0:q1, j].double() @ K.t().contiguous()) / math.sqrt(D)
                e.masked_fill_(~seen, -math.inf)
                lse = torch.logsumexp(e, dim=1, keepdim=True)
                p = torch.exp(e - lse)
                p[~seen.any(dim=1)] = 0.0
                out[q0:q1, j] = p @ V
    return out
