"""Timed cases of the attention-layer operators: position rotation over one
to four axes, the append of keys and values to a paged cache, and attention
of new tokens over that cache.

Around the 1-bit projections of pq1 an attention layer does three more
things: it rotates queries and keys by their positions, it stores the new keys
and values in a paged cache, and it attends over that cache.  The cases here
are those three steps at the sizes serving meets, with the head shapes of the
tested 27B model (24 query heads, 4 key heads, 256 wide, 64 of them rotated
over time, height and width) next to generic ones.

``own`` False computes each operator from elementary torch operations in 32
bits (angles in 64); ``own`` True calls the library.
"""
import math
import random

import torch

own = False

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
_DT = {"f32": F32, "bf16": BF16, "f16": F16}
_BASE = 1.0e6  # frequency base of the rotation


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _rope(name, T, H, D, rot, sections, pairing, interleaved, inverse, din, dout, far):
    return {"name": name, "op": "rope", "T": T, "H": H, "D": D, "rot": rot, "sections": sections,
            "pairing": pairing, "interleaved": interleaved, "inverse": inverse, "din": din,
            "dout": dout, "far": far}


def _append(name, T, B, pad, Hk, G, D, rot, sections, pairing, interleaved, page, din, dtype, far):
    return {"name": name, "op": "append", "T": T, "B": B, "pad": pad, "Hk": Hk, "G": G, "D": D,
            "rot": rot, "sections": sections, "pairing": pairing, "interleaved": interleaved,
            "page": page, "din": din, "dtype": dtype, "far": far}


def _attention(name, B, q_min, q_max, past_min, past_max, Hk, G, D, page, dtype, dout, causal,
               window):
    return {"name": name, "op": "attention", "B": B, "q_min": q_min, "q_max": q_max,
            "past_min": past_min, "past_max": past_max, "Hk": Hk, "G": G, "D": D, "page": page,
            "dtype": dtype, "dout": dout, "causal": causal, "window": window}


def listed():
    return [
        # the query of one decoded token, straight from the fp32 projection
        _rope("rope one token", 1, 24, 256, 64, "11,11,10", "halves", True, False, "f32", "bf16",
              5000),
        # a 37 x 37 patch image in a vision encoder: every element rotated, height and width
        _rope("rope image patches", 1369, 16, 72, 72, "18,18", "halves", False, False, "bf16",
              "bf16", 0),
        # gradient of the queries of a long training sequence (the rotation run backwards)
        _rope("rope gradient", 8190, 24, 256, 64, "11,11,10", "halves", True, True, "bf16",
              "bf16", 0),
        # one user decoding: query and key rotated, key and value stored
        _append("append one token", 1, 1, 0, 4, 6, 256, 64, "11,11,10", "halves", True, 16, "f32",
                "bf16", 9000),
        # a batch of users decoding, the batch padded to a fixed size
        _append("append decode batch", 96, 91, 5, 8, 4, 128, 128, "64", "halves", False, 32,
                "f16", "f16", 20000),
        # three prompts entering the cache together
        _append("append prompts", 4001, 3, 0, 4, 6, 256, 64, "11,11,10", "halves", True, 64,
                "f32", "bf16", 0),
        # one user early in a conversation; fp32 out for the rotation of the output projection
        _attention("attend one token", 1, 1, 1, 700, 700, 4, 6, 256, 16, "bf16", "f32", True, 0),
        # a batch of users decoding at their own lengths
        _attention("attend decode batch", 64, 1, 1, 200, 8000, 4, 6, 256, 64, "bf16", "bf16",
                   True, 0),
        # one user far into a long document
        _attention("attend long context", 1, 1, 1, 131070, 131070, 4, 6, 256, 256, "bf16", "f32",
                   True, 0),
        # a few drafted tokens for each user are verified, sliding window
        _attention("attend drafts", 16, 2, 6, 500, 4000, 8, 4, 128, 32, "f16", "f16", True, 1024),
        # a chunk of a long prompt after the part already in the cache
        _attention("attend prompt chunk", 1, 2048, 2048, 6144, 6144, 4, 6, 256, 64, "bf16",
                   "bf16", True, 0),
        # whole prompts of ragged lengths
        _attention("attend prompts", 5, 30, 4000, 0, 0, 8, 4, 128, 16, "bf16", "bf16", True, 0),
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
    kind = rng.choice(["rope", "append", "attention", "attention"])
    if kind == "rope":
        D = rng.choice([64, 72, 80, 96, 128, 128, 256])
        H = rng.choice([1, 4, 8, 16, 24, 32])
        T = _log(rng, 1, min(8000, 48_000_000 // (H * D)))
        rot, sec, inter = _draw_rotation(rng, D, rng.random() < 0.5)
        c = _rope("", T, H, D, rot, sec, rng.choice(["halves", "halves", "adjacent"]), inter,
                  rng.random() < 0.3, rng.choice(["f32", "bf16", "f16"]), None,
                  rng.choice([0, 0, 10000, 500000]))
        c["dout"] = rng.choice([c["din"], {"f32": "bf16"}.get(c["din"], c["din"])])
    elif kind == "append":
        D = rng.choice([64, 80, 128, 256])
        Hk, G = rng.choice([(1, 8), (2, 7), (4, 6), (4, 6), (8, 4), (8, 1), (4, 0)])
        T = _log(rng, 1, min(4000, 30_000_000 // ((2 + G) * Hk * D)))
        B = rng.choice([1, max(1, T // 100), min(T, 64)])
        rot, sec, inter = _draw_rotation(rng, D, rng.random() < 0.5)
        if G == 0 and rng.random() < 0.5:
            rot, sec, inter = 0, "", False
        pad = 0 if T < 4 else rng.choice([0, 0, min(3, T - B)])
        dt = rng.choice(["bf16", "f16"])
        c = _append("", T, B, pad, Hk, G, D, rot, sec, rng.choice(["halves", "adjacent"]), inter,
                    rng.choice([1, 8, 16, 32, 64, 128]), rng.choice(["f32", dt]), dt,
                    rng.choice([0, 10000, 500000]))
    else:
        D = rng.choice([64, 128, 256])
        Hk, G = rng.choice([(1, 8), (2, 7), (4, 6), (4, 6), (8, 4), (8, 1), (2, 16)])
        shape = rng.choice(["decode", "decode", "drafts", "chunk", "prompt"])
        q_max = {"decode": 1, "drafts": rng.randint(2, 8), "chunk": _log(rng, 9, 2000),
                 "prompt": _log(rng, 2, 4000)}[shape]
        q_min = q_max if rng.random() < 0.5 else rng.randint(1, q_max)
        past = 0 if shape == "prompt" else _log(rng, 1, 60000 if shape == "decode" else 8000)
        B = _log(rng, 1, 64)
        window = rng.choice([0, 0, 0, rng.randint(1, 4000)])
        causal = True if window else rng.random() < 0.85
        dt = rng.choice(["bf16", "bf16", "f16"])
        c = _attention("", B, q_min, q_max, rng.randint(0, past), past, Hk, G, D,
                       rng.choice([1, 8, 16, 32, 64, 128, 256]), dt,
                       rng.choice([dt, dt, "f32"]), causal, window)
        # no more than the largest listed cases, in products and in bytes
        while c["B"] > 1 and (work(c)["flops"] > 2.5e11 or work(c)["bytes"] > 5.0e8):
            c["B"] = c["B"] // 2
        while work(c)["flops"] > 2.5e11 or work(c)["bytes"] > 5.0e8:
            c["q_max"] = max(1, c["q_max"] // 2)
            c["q_min"] = min(c["q_min"], c["q_max"])
            c["past_max"] //= 2
            c["past_min"] = min(c["past_min"], c["past_max"])
    del c["name"]
    return c


def _lens(case):
    """New tokens and cached tokens of every sequence: a function of the case
    alone, so that its work is known without its inputs."""
    rng = random.Random(case["B"] * 1000003 + case["q_max"] * 1009 + case["past_max"])
    q = [rng.randint(case["q_min"], case["q_max"]) for _ in range(case["B"])]
    past = [rng.randint(case["past_min"], case["past_max"]) for _ in range(case["B"])]
    q[0] = case["q_max"]
    past[0] = case["past_max"]
    return q, past


def _visible(case, n, past):
    """(query, key) pairs of one sequence that the mask leaves, and its keys that are read."""
    kv = n + past
    if not case["causal"]:
        return n * kv, kv
    w = case["window"] or kv
    # row i sees min(w, past + i + 1) keys
    full = max(0, min(n, w - past))           # rows whose window reaches the first key
    pairs = full * past + full * (full + 1) // 2 + (n - full) * w
    return pairs, kv - max(0, past + 1 - w)


def work(case):
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if case["op"] == "rope":
        n = case["T"] * case["H"] * case["D"]
        axes = len(case["sections"].split(","))
        return {"bytes": n * (size[case["din"]] + size[case["dout"]]) + 4 * axes * case["T"]
                + 4 * case["rot"], "flops": 3 * case["T"] * case["H"] * case["rot"]}
    if case["op"] == "append":
        T, live = case["T"], case["T"] - case["pad"]
        kv, q = 2 * case["Hk"] * case["D"], case["Hk"] * case["G"] * case["D"]
        axes = len(case["sections"].split(",")) if case["rot"] else 0
        io = size[case["din"]] + size[case["dtype"]]
        return {"bytes": live * kv * io + T * q * io + T * (8 + 4 * axes) + 4 * case["rot"],
                "flops": 3 * T * case["Hk"] * (1 + case["G"]) * case["rot"]}
    qs, pasts = _lens(case)
    Hq = case["Hk"] * case["G"]
    pairs = keys = pages = 0
    for n, p in zip(qs, pasts):
        a, b = _visible(case, n, p)
        pairs, keys, pages = pairs + a, keys + b, pages + -(-b // case["page"])
    rows = sum(qs) * Hq
    return {"bytes": rows * case["D"] * (2 + size[case["dout"]]) + keys * case["Hk"] * case["D"] * 4
            + 4 * pages + 4 * (2 * case["B"] + 1), "flops": 4 * pairs * Hq * case["D"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


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


def _inputs(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        s["x"] = torch.randn(T, H, D, device="cuda", generator=g).to(_DT[case["din"]])
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
        shape = (pages, Hk, page, D)
        s["k_cache"] = torch.randn(shape, device="cuda", generator=g).to(_DT[case["dtype"]])
        s["v_cache"] = torch.randn(shape, device="cuda", generator=g).to(_DT[case["dtype"]])
        if case["rot"]:
            s["positions"] = _positions(case, T, g)
            s["freqs"] = _freqs(case["rot"])
    else:
        Hk, G, D, page = (case[k] for k in ("Hk", "G", "D", "page"))
        qs, pasts = _lens(case)
        dt = _DT[case["dtype"]]
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
        s["q"] = (1.5 * torch.randn(sum(qs), Hk * G, D, device="cuda", generator=g)).to(dt)
        s["k_cache"] = torch.randn((pages, Hk, page, D), device="cuda", generator=g).to(dt)
        s["v_cache"] = torch.randn((pages, Hk, page, D), device="cuda", generator=g).to(dt)
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
        if case["op"] != "attention" and case["rot"]:
            s["rope"] = pq1.Rope(case["rot"], _sections(case), freqs=s["freqs"],
                                 pairing=case["pairing"], interleaved=case["interleaved"])
        if case["op"] != "rope":
            s["cache"] = pq1.KVCache(s["k_cache"], s["v_cache"])
    elif case["op"] != "attention" and case["rot"]:
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
    if case["op"] == "rope":
        return pq1.pq1_rope(s["x"], s["positions"], s["rope"], out_dtype=_DT[case["dout"]],
                            inverse=case["inverse"])
    if case["op"] == "append":
        q_out = pq1.pq1_kv_append(s["cache"], s["k"], s["v"], s["slots"],
                                  positions=s.get("positions"), rope=s.get("rope"), q=s["q"])
        out = (s["k_cache"], s["v_cache"])
        return out if q_out is None else out + (q_out,)
    return pq1.pq1_paged_attention(s["q"], s["cache"], s["table"], s["cu"], s["kv"],
                                   max_q=s["max_q"], max_kv=s["max_kv"], causal=case["causal"],
                                   window=case["window"], out_dtype=_DT[case["dout"]])


def _rotate_plain(x, s, inverse):
    """x [T][H][D] in 32 bits, rotated; angles in 64 bits, reduced before they are narrowed."""
    case = s["case"]
    rot = case["rot"]
    angle = s["positions"].double()[s["axis"]].t() * s["freqs"]
    angle = torch.remainder(angle, 2.0 * math.pi).float().unsqueeze(1)
    c, n = torch.cos(angle), torch.sin(angle)
    if inverse:
        n = -n
    x = x.float()
    y = x.clone()
    if case["pairing"] == "halves":
        lo, hi = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        lo, hi = slice(0, rot, 2), slice(1, rot, 2)
    y[..., lo] = x[..., lo] * c - x[..., hi] * n
    y[..., hi] = x[..., hi] * c + x[..., lo] * n
    return y


def _run_plain(s):
    case = s["case"]
    if case["op"] == "rope":
        return _rotate_plain(s["x"], s, case["inverse"]).to(_DT[case["dout"]])
    if case["op"] == "append":
        dt, page = _DT[case["dtype"]], case["page"]
        k, v = s["k"].float(), s["v"]
        if case["rot"]:
            k = _rotate_plain(k, s, False)
        live = torch.nonzero(s["slots"] >= 0).squeeze(1)
        at = s["slots"][live]
        s["k_cache"][at // page, :, at % page] = k[live].to(dt)
        s["v_cache"][at // page, :, at % page] = v[live].to(dt)
        out = (s["k_cache"], s["v_cache"])
        if s["q"] is None:
            return out
        q = _rotate_plain(s["q"], s, False) if case["rot"] else s["q"]
        return out + (q.to(dt),)
    Hk, G, D, page = (case[k] for k in ("Hk", "G", "D", "page"))
    out = torch.zeros(s["q"].shape, dtype=_DT[case["dout"]], device="cuda")
    for b in range(case["B"]):
        q0, q1, kv = s["cu_host"][b], s["cu_host"][b + 1], s["kv_host"][b]
        n = q1 - q0
        key = torch.arange(kv, device="cuda")
        where, off = s["table"][b, key // page].long(), key % page
        K = s["k_cache"][where, :, off].float().permute(1, 2, 0).contiguous()   # [Hk][D][kv]
        V = s["v_cache"][where, :, off].float().permute(1, 0, 2).contiguous()   # [Hk][kv][D]
        q = s["q"][q0:q1].float().view(n, Hk, G, D).permute(1, 2, 0, 3).reshape(Hk, G * n, D)
        score = torch.matmul(q, K).view(Hk, G, n, kv) * (1.0 / math.sqrt(D))
        if case["causal"]:
            at = torch.arange(n, device="cuda").unsqueeze(1) + (kv - n)
            hidden = key > at
            if case["window"]:
                hidden = hidden | (key <= at - case["window"])
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
def _rotate_exact(x, positions, case, inverse):
    """Each pair as a complex number times exp(i pos f)."""
    rot, half = case["rot"], case["rot"] // 2
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
    x = x.double()
    head = x[..., :rot]
    if case["pairing"] == "halves":
        w = torch.complex(head[..., :half], head[..., half:]) * z
        turned = torch.cat([w.real, w.imag], dim=-1)
    else:
        w = torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * z
        turned = torch.view_as_real(w).flatten(-2)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        return _rotate_exact(s["x"], s["positions"], case, case["inverse"])
    if case["op"] == "append":
        turn = (lambda x: _rotate_exact(x, s["positions"], case, False)) if case["rot"] \
            else (lambda x: x.double())
        # slot-major view of the caches: [pages * page][Hk][D]
        out = []
        for cache, new in ((s["k_cache"], turn(s["k"])), (s["v_cache"], s["v"].double())):
            flat = cache.double().transpose(1, 2).reshape(-1, case["Hk"], case["D"])
            used = s["slots"] >= 0
            flat.index_copy_(0, s["slots"][used], new[used])
            out.append(flat.view(cache.shape[0], case["page"], case["Hk"], case["D"])
                       .transpose(1, 2).contiguous())
        return tuple(out) if s["q"] is None else (*out, turn(s["q"]))
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
                seen = seen.triu(kv - n - case["window"] + 1)
        for h in range(Hk):
            K = s["k_cache"][rows, h].reshape(-1, D)[:kv].double()
            V = s["v_cache"][rows, h].reshape(-1, D)[:kv].double()
            for j in range(h * G, (h + 1) * G):
                e = (s["q"][q0:q1, j].double() @ K.t().contiguous()) / math.sqrt(D)
                e.masked_fill_(~seen, -math.inf)
                lse = torch.logsumexp(e, dim=1, keepdim=True)
                p = torch.exp(e - lse)
                p[~seen.any(dim=1)] = 0.0
                out[q0:q1, j] = p @ V
    return out
