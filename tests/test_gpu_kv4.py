"""Norms of heads with the rotation, and the 4-bit cache's append and read, on the
GPU against their 64-bit forms."""
import math

import pytest
import torch

import attention_reference as ref
import kv4_reference as ref4
from test_gpu_attention import check, positions_of

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pq(dev):
    from gemm_hadamard_rotated_amd import pq1
    pq1.load_library()
    return pq1


def rotation(pq, dev, rot, sections, pairing, inter, base=1.0e4):
    """The Rope and the reference's arguments after the positions; (None, {}) for none."""
    if not rot:
        return None, {}
    freqs = pq.rope_frequencies(rot, base)
    rope = pq.Rope(rot, sections, freqs=freqs.to(dev), pairing=pairing, interleaved=inter)
    return rope, dict(freqs=freqs, sections=sections, pairing=pairing, interleaved=inter)


def drawn(shape, seed, dtype=F32, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(shape, generator=g)).to(dtype)


# ---------------------------------------------------------------------------
# Norm and rotation
# ---------------------------------------------------------------------------
NORM = [
    # T, H, D, rot, sections, pairing, interleaved, in, out, first position
    (1, 24, 256, 64, (11, 11, 10), "halves", True, F32, BF16, 5000),
    (1, 1, 8, 2, (1,), "adjacent", False, F32, F32, 0),
    (7, 3, 72, 72, (18, 18), "halves", False, BF16, BF16, 0),
    (130, 5, 80, 20, (4, 3, 3), "adjacent", False, F16, F32, 9),
    (33, 4, 64, 64, (32,), "halves", False, BF16, F16, 2 ** 31 - 40),
    (33, 4, 128, 128, (16, 24, 24), "halves", False, F16, F16, -70000),
    (260, 2, 96, 48, (6, 6, 6, 6), "adjacent", True, F32, F32, 1000000),
    (9, 2, 40, 22, (11,), "halves", False, F32, F16, 3),
    (5, 1024, 16, 16, (0, 8), "halves", False, BF16, F32, 77),
    (20000, 1, 64, 32, (16,), "halves", False, BF16, BF16, 0),
    (3, 2, 1024, 1024, (512,), "adjacent", False, F32, BF16, 12),
    (4, 3, 1024, 1024, (512,), "halves", False, BF16, F32, 12),
    (5, 2, 520, 516, (258,), "halves", False, F32, F32, 3),       # eights past 512, odd halves
    (6, 2, 512, 128, (64,), "halves", False, F16, BF16, 3),
    (301, 8, 72, 18, (9,), "halves", False, BF16, BF16, 0),
    (50, 3, 24, 18, (9,), "adjacent", False, F32, F16, 0),
    (40, 7, 128, 0, (), "halves", False, BF16, F32, 0),            # no rotation
    (2, 2, 1016, 0, (), "halves", False, F32, F32, 0),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", NORM, ids=lambda c: "-".join(str(v) for v in c[:4]))
def test_norm_rope(pq, dev, case, inverse):
    T, H, D, rot, sections, pairing, inter, din, dout, first = case
    x = drawn((T, H, D), T * 31 + D, din, 3.0)
    w = 1 + drawn((D,), 5, F32, 0.3)
    pos = positions_of(T, max(1, len(sections)), first, T)
    rope, more = rotation(pq, dev, rot, sections, pairing, inter)
    y = pq.pq1_norm_rope(x.to(dev), w.to(dev), pos.to(dev), rope, eps=1e-5, out_dtype=dout,
                         inverse=inverse)
    assert y.dtype == dout and y.is_contiguous()
    e, b = ref4.norm_rope(x, w, 1e-5, pos, inverse=inverse, **more)
    check(y, e, ref.rounded_bound(e, b, dout), "norm")


def test_norm_of_any_size_of_head(pq, dev):
    """No finite head over- or underflows; zeros stay; infinities and NaN as the formula says."""
    D = 128
    x = drawn((12, 2, D), 3)
    for i, size in enumerate((1e-44, 1e-38, 1e-30, 1e-20, 1e-3, 1.0, 1e10, 1e19, 1e30, 5e37)):
        x[i] *= size
    x[10] = 0.0
    x[11, 0] = torch.full((D,), torch.finfo(F32).max)
    w = 1 + drawn((D,), 4, F32, 0.3)
    for eps in (1e-6, 1e-30, 2.0 ** -149, 3e38):
        eps32 = float(torch.tensor(eps, dtype=F32))
        y = pq.pq1_norm_rope(x.to(dev), w.to(dev), eps=eps)
        e, b = ref4.norm_rope(x, w, eps32)
        check(y, e, ref.rounded_bound(e, b, F32), f"eps {eps}")
    x = drawn((3, 2, D), 3)
    x[0, 0, 7] = math.inf
    x[1, 1, 100] = -math.inf
    x[2, 0, 3] = math.nan
    y = pq.pq1_norm_rope(x.to(dev), w.to(dev), eps=1e-6).cpu()
    assert torch.isnan(y[0, 0, 7]) and torch.isnan(y[1, 1, 100]) and torch.isnan(y[2, 0]).all()
    assert int(torch.isnan(y).sum()) == D + 2
    rest = torch.ones(D, dtype=torch.bool)
    rest[7] = False
    assert (y[0, 0][rest] == 0).all()
    e, b = ref4.norm_rope(x[1:2, :1], w, 1e-6)
    check(y[1:2, :1], e, ref.rounded_bound(e, b, F32), "a neighbour of an infinite head")


def test_norm_strided_and_in_place(pq, dev):
    T, H, D, rot = 37, 3, 64, 32
    stacked = drawn((T, 5 * D * H), 5).to(dev)
    x = stacked[:, D * H:2 * D * H].unflatten(1, (H, D))
    w = 1 + drawn((D,), 6, F32, 0.3)
    pos = positions_of(T, 1, 100, 3)
    rope, more = rotation(pq, dev, rot, (16,), "halves", False)
    x0, before = x.cpu().clone(), stacked.clone()
    e, b = ref4.norm_rope(x0, w, 1e-6, pos, **more)
    check(pq.pq1_norm_rope(x, w.to(dev), pos.to(dev)[0], rope), e, ref.rounded_bound(e, b, F32), "strided")
    heads_first = drawn((H, T, D), 8).to(dev).transpose(0, 1)
    out = torch.empty(T, H, 2 * D, device=dev)[..., :D]
    assert pq.pq1_norm_rope(heads_first, w.to(dev), pos.to(dev), rope, out=out) is out
    e2, b2 = ref4.norm_rope(heads_first.cpu(), w, 1e-6, pos, **more)
    check(out, e2, ref.rounded_bound(e2, b2, F32), "heads first")
    pq.pq1_norm_rope(x, w.to(dev), pos.to(dev), rope, out=x)
    check(x, e, ref.rounded_bound(e, b, F32), "in place")
    assert torch.equal(stacked[:, :D * H], before[:, :D * H])
    assert torch.equal(stacked[:, 2 * D * H:], before[:, 2 * D * H:])
    assert pq.pq1_norm_rope(x[:0], w.to(dev), pos.to(dev)[:, :0].contiguous(), rope).shape == (0, H, D)


GRAD = [c for c in NORM if c[0] < 1000] + [
    (2500, 3, 64, 64, (32,), "halves", False, BF16, BF16, 0),      # more groups than workgroups
    (9000, 1, 256, 64, (11, 11, 10), "halves", True, BF16, F32, 0),
]


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", GRAD, ids=lambda c: "-".join(str(v) for v in c[:4]))
def test_norm_rope_grad(pq, dev, case, inverse):
    T, H, D, rot, sections, pairing, inter, din, dg, first = case
    x, g = drawn((T, H, D), T * 31 + D, din, 3.0), drawn((T, H, D), 77, dg)
    w = 1 + drawn((D,), 5, F32, 0.3)
    pos = positions_of(T, max(1, len(sections)), first, T)
    rope, more = rotation(pq, dev, rot, sections, pairing, inter)
    call = lambda **kw: pq.pq1_norm_rope_grad(g.to(dev), x.to(dev), w.to(dev), pos.to(dev), rope,
                                              eps=1e-5, inverse=inverse, **kw)
    dx, dw = call()
    assert dx.dtype == din and dw.dtype == F32
    ex, bx, ew, bw = ref4.norm_rope_grad(g, x, w, 1e-5, pos, inverse=inverse, **more)
    check(dx, ex, ref.rounded_bound(ex, bx, din), "dx")
    check(dw, ew, bw, "dw")
    again = call()
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw), "the same from run to run"
    alone = call(weight_grad=False)
    assert alone[1] is None and torch.equal(alone[0], dx)


def test_norm_rope_grad_against_differences(pq, dev):
    """d/dh of sum(g * y(x + h d)) and of weights, by central differences in 64 bits."""
    T, H, D, rot = 3, 2, 64, 32
    x, g, d = drawn((T, H, D), 1), drawn((T, H, D), 2), drawn((T, H, D), 3)
    w, dw = 1 + drawn((D,), 4, F32, 0.3), drawn((D,), 5)
    pos = positions_of(T, 1, 50, 3)
    rope, more = rotation(pq, dev, rot, (16,), "halves", False)
    gx, gw = pq.pq1_norm_rope_grad(g.to(dev), x.to(dev), w.to(dev), pos.to(dev), rope)
    f = lambda x, w: float((ref4.norm_rope(x, w, 1e-6, pos, **more)[0] * g.double()).sum())
    h = 1e-5
    by_x = (f(x.double() + h * d.double(), w) - f(x.double() - h * d.double(), w)) / (2 * h)
    by_w = (f(x, w.double() + h * dw.double()) - f(x, w.double() - h * dw.double())) / (2 * h)
    # differences are off by h^2 of third derivatives and 2^-52 / h of the sum, results by 2^-20
    assert abs(float((gx.double().cpu() * d.double()).sum()) - by_x) <= 1e-4
    assert abs(float((gw.double().cpu() * dw.double()).sum()) - by_w) <= 1e-4


def test_norm_rope_grad_in_place_and_empty(pq, dev):
    T, H, D = 50, 2, 96
    x, g = drawn((T, H, D), 1).to(dev), drawn((T, H, D), 2).to(dev)
    w = (1 + drawn((D,), 4, F32, 0.3)).to(dev)
    dx, dw = pq.pq1_norm_rope_grad(g, x, w)
    for which in (0, 1):
        a, b = x.clone(), g.clone()
        got = pq.pq1_norm_rope_grad(b, a, w, dx=(a, b)[which])
        assert got[0] is (a, b)[which] and torch.equal(got[0], dx) and torch.equal(got[1], dw)
    dx, dw = pq.pq1_norm_rope_grad(g[:0], x[:0], w)
    assert dx.shape == (0, H, D) and torch.equal(dw, torch.zeros_like(w))
    tiny = x * 1e-30                       # r at its limit, eps^(-1/2)
    dx, dw = pq.pq1_norm_rope_grad(g, tiny, w)
    ex, bx, ew, bw = ref4.norm_rope_grad(g.cpu(), tiny.cpu(), w.cpu(), 1e-6)
    check(dx, ex, ref.rounded_bound(ex, bx, F32), "tiny heads")
    check(dw, ew, bw, "tiny heads' weights")


# ---------------------------------------------------------------------------
# The 4-bit cache
# ---------------------------------------------------------------------------
def filled(pq, dev, pages, page, heads, dim, dtype, seed=0):
    """A cache of arbitrary bytes, as a recycled one holds."""
    g = torch.Generator().manual_seed(seed)
    c = pq.KV4Cache.empty(pages, page, heads, dim, dtype, dev)
    for t in (c.k, c.k_scale, c.v, c.v_scale):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, dtype=torch.uint8))
    return c


def rows(t, slots, page):
    """[pages][heads][page][n] at slots: [T][heads][n]."""
    return t.cpu()[slots // page, :, slots % page]


APPEND4 = [
    # T, Hk, G, D, page, rot, sections, pairing, interleaved, in, dtype, norms
    (1, 4, 6, 256, 16, 64, (11, 11, 10), "halves", True, F32, BF16, "kq"),
    (91, 8, 4, 128, 32, 128, (64,), "halves", False, F16, F16, "kq"),
    (33, 1, 8, 64, 1, 64, (32,), "adjacent", False, BF16, BF16, "k"),
    (300, 2, 7, 96, 8, 20, (10,), "halves", False, F32, F16, "q"),
    (50, 4, 0, 64, 128, 64, (8, 12, 12), "adjacent", False, BF16, BF16, "k"),
    (21, 3, 2, 32, 4, 0, (), "halves", False, F32, BF16, ""),
    (40, 2, 2, 32, 4, 0, (), "halves", False, BF16, BF16, "kq"),
    (12, 2, 1, 544, 2, 540, (270,), "halves", False, F32, BF16, "kq"),   # eights past 512
    (3, 1, 1, 1024, 1, 1024, (512,), "halves", False, F32, BF16, "kq"),
    (7, 1, 2, 1024, 1, 64, (32,), "adjacent", False, BF16, BF16, ""),
    (1500, 4, 2, 128, 64, 64, (32,), "halves", False, BF16, BF16, "kq"),
]


@pytest.mark.parametrize("kind", ["4 bits", "16 bits"])
@pytest.mark.parametrize("case", APPEND4, ids=lambda c: "-".join(str(v) for v in (*c[:6], c[11])))
def test_append_with_norms(pq, dev, case, kind):
    T, Hk, G, D, page, rot, sections, pairing, inter, din, dt, norms = case
    if kind == "16 bits" and not norms:
        pytest.skip("that append is without norms")
    Hq = Hk * G
    pages = -(-T // page) + 3
    qkv = drawn((T, (Hq + 2 * Hk) * D), T + D, din)
    q = qkv[:, :Hq * D].unflatten(1, (Hq, D)) if G else None
    k = qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    v = qkv[:, (Hq + Hk) * D:].unflatten(1, (Hk, D))
    gpu = qkv.to(dev)
    gq, gk, gv = (None if t is None else gpu[:, t.storage_offset():t.storage_offset() + t.shape[1] * D]
                  .unflatten(1, (t.shape[1], D)) for t in (q, k, v))
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 4:
        slots[T // 2] = -1
        slots[1] = pages * page              # past the cache: not stored either
    pos = positions_of(T, max(1, len(sections)), 1000, T)
    rope, more = rotation(pq, dev, rot, sections, pairing, inter, 1.0e6)
    kw, qw = (1 + drawn((D,), s, F32, 0.3) if name in norms else None for s, name in ((8, "k"), (9, "q")))
    norm = pq.HeadNorm(*(None if t is None else t.to(dev) for t in (kw, qw)), eps=1e-6) if norms else None
    if kind == "4 bits":
        cache = filled(pq, dev, pages, page, Hk, D, dt)
        held = (cache.k, cache.k_scale, cache.v, cache.v_scale)
        call = pq.pq1_kv4_append
    else:
        cache = pq.KVCache(*(drawn((pages, Hk, page, D), s, dt).to(dev) for s in (1, 2)))
        held = (cache.k, cache.v)
        call = pq.pq1_kv_append
    before = [t.clone().cpu() for t in held]
    out = call(cache, gk, gv, slots.to(dev), positions=pos.to(dev), rope=rope, q=gq, norm=norm)
    live = (slots >= 0) & (slots < pages * page)
    at = slots[live]
    # keys and values
    kz = k.double()
    if kw is not None:
        kz = kz * ref4.root(k, 1e-6) * kw.double()
    if rot:
        kz, kb = ref.rotate(kz, pos, more["freqs"], sections, pairing, inter)
    if kind == "4 bits":
        for name, x, codes, scales in (("k", kz, held[0], held[1]), ("v", v.double(), held[2], held[3])):
            want, byte = ref4.quantise(x[live], dt)
            assert torch.equal(rows(scales, at, page), byte), f"{name}: scales"
            got = ref4.values(rows(codes, at, page), rows(scales, at, page))
            assert torch.equal(got, want), f"{name}: {int((got != want).sum())} values"
    else:
        if kw is not None:
            e, b = ref4.norm_rope(k, kw, 1e-6, pos, **more)
        else:
            e, b = (kz, kb) if rot else (kz, torch.zeros_like(kz))
        check(rows(held[0], at, page), e[live], ref.rounded_bound(e, b, dt)[live], "k")
        assert torch.equal(rows(held[1], at, page), v[live].to(dt))
    # every other row is as it was
    untouched = torch.ones(pages * page, dtype=torch.bool)
    untouched[at] = False
    other = torch.nonzero(untouched).squeeze(1)
    for t, old in zip(held, before):
        assert torch.equal(rows(t, other, page), rows(old, other, page)), "other rows"
    if q is None:
        assert out is None
        return
    if qw is not None:
        e, b = ref4.norm_rope(q, qw, 1e-6, pos, **more)
    elif rot:
        e, b = ref.rotate(q, pos, more["freqs"], sections, pairing, inter)
    else:
        e, b = q.double(), torch.zeros_like(q, dtype=torch.float64)
    assert out.dtype == dt
    check(out, e, ref.rounded_bound(e, b, dt), "q")


@pytest.mark.parametrize("din", ["f32", "cache"])
@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
def test_append4_of_borders_and_extremes(pq, dev, dt, din):
    """Values on, just under and just over every border, groups of every size, infinities."""
    kind = F32 if din == "f32" else dt
    grid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 0.0, 0.5, 1, 1.5, 2, 3, 4],
                        dtype=torch.float64)
    groups = []
    sizes = range(-130, 126) if dt == BF16 else range(-28, 16)
    for n in sizes:
        unit = 2.0 ** n
        for top in (7.0, 6.0, 6.9, 3.6, 7.1):
            g = torch.zeros(32, dtype=torch.float64)
            g[:16] = grid * unit
            g[16:24] = torch.nextafter(grid[:8].float(), torch.tensor(9.0)).double() * unit
            g[24:31] = -torch.nextafter(grid[:7].float(), torch.tensor(0.0)).double() * unit
            g[g.abs() > top * unit] = 0
            g[31] = -top * unit
            groups.append(g)
    x = torch.stack(groups).to(F32).to(kind)
    odd = torch.zeros(8, 32)
    odd[0, 3] = math.inf
    odd[1, 31] = -math.inf
    odd[2, 0] = math.nan
    odd[3, 5] = -0.0
    odd[4] = torch.finfo(kind).max
    odd[5] = torch.finfo(kind).tiny
    odd[6, 9] = -torch.finfo(kind).max
    odd[6, 10] = math.nan
    x = torch.cat([x, odd.to(kind)])
    x = torch.cat([x, x.new_zeros((-x.shape[0]) % 4, 32)]).view(-1, 1, 128)
    T = x.shape[0]
    cache = filled(pq, dev, -(-T // 8), 8, 1, 128, dt)
    pq.pq1_kv4_append(cache, x.to(dev), x.flip(0).to(dev), torch.arange(T, device=dev))
    at = torch.arange(T)
    for codes, scales, src in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, x.flip(0))):
        want, byte = ref4.quantise(src, dt)
        assert torch.equal(rows(scales, at, 8), byte)
        got = ref4.values(rows(codes, at, 8), rows(scales, at, 8))
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        fine = ~torch.isnan(want)
        assert torch.equal(got[fine], want[fine])
    bad = ~torch.isfinite(x.view(-1, 32)).all(dim=1)     # 2^15 times 7 among them, in f16
    assert int(torch.isnan(want).sum()) == 32 * int(bad.sum()) >= 32 * 4
    # what it holds is a number of the cache's type, exactly
    k, v = pq.pq1_kv4_read(cache, torch.arange(T, device=dev))
    assert k.dtype == dt
    assert torch.equal(v.double().cpu()[fine], want[fine])


def test_append4_next_to_a_border_after_the_norm(pq, dev):
    """A key whose normalised value lies closer to a border than fp32 resolves: its
    code is that of the 64-bit value."""
    D = 64
    x = torch.ones(400, 1, D)
    x[:, 0, 0] = 7.0
    # around 1.25 of a unit: with the weight below some land just under it, some over
    x[:, 0, 1] = 1.25 * (1 + (torch.arange(400) - 200) * 2.0 ** -23)
    x = x.to(dev)
    w = torch.ones(D)
    r = float(ref4.root(x[200:201].cpu(), 1e-6))
    w[:] = float(torch.tensor(0.5 / r, dtype=F32))          # units near a power of two
    cache = filled(pq, dev, 50, 8, 1, D, BF16)
    pq.pq1_kv4_append(cache, x, x, torch.arange(400, device=dev),
                      norm=pq.HeadNorm(w.to(dev), eps=1e-6))
    want, byte = ref4.quantise(x.cpu().double() * ref4.root(x.cpu(), float(torch.tensor(1e-6))) * w.double(), BF16)
    at = torch.arange(400)
    assert torch.equal(rows(cache.k_scale, at, 8), byte)
    assert torch.equal(ref4.values(rows(cache.k, at, 8), rows(cache.k_scale, at, 8)), want)


READ4 = [
    # T, H, D, page, dtype, out
    (1, 4, 256, 16, BF16, BF16),
    (333, 2, 64, 1, F16, F16),
    (700, 1, 32, 8, BF16, F32),
    (50, 3, 96, 32, F16, F32),
    (9, 1, 1024, 4, BF16, BF16),
]


@pytest.mark.parametrize("case", READ4, ids=lambda c: "-".join(str(v) for v in c[:4]))
def test_read4(pq, dev, case):
    T, H, D, page, dt, dout = case
    pages = -(-T // page) + 2
    cache = filled(pq, dev, pages, page, H, D, dt, 3)
    g = torch.Generator().manual_seed(T)
    lo, hi = ref4.EXPONENTS[dt]
    for s in (cache.k_scale, cache.v_scale):     # scales the append gives, and NaN
        s.copy_(torch.randint(max(lo, -60) + 127, min(hi, 60) + 128, s.shape, generator=g, dtype=torch.uint8))
        s.view(-1)[::7] = 255
    slots = torch.randint(0, pages * page, (T,), generator=g)    # some of them twice
    if T > 2:
        slots[1], slots[2] = -1, pages * page
    k, v = pq.pq1_kv4_read(cache, slots.to(dev), out_dtype=dout)
    live = (slots >= 0) & (slots < pages * page)
    for got, codes, scales in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        assert got.dtype == dout and got.shape == (T, H, D)
        want = torch.zeros(T, H, D, dtype=torch.float64)
        want[live] = ref4.values(rows(codes, slots[live], page), rows(scales, slots[live], page))
        got = got.double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got.nan_to_num(0), want.nan_to_num(0))
    # one of the two, into slices
    wide = torch.full((T, H, 2, D), 7.0, dtype=dout, device=dev)
    only = pq.pq1_kv4_read(cache, slots.to(dev), v_out=wide[:, :, 1])
    assert only[0] is None and torch.equal(only[1].nan_to_num(0), v.nan_to_num(0))
    assert (wide[:, :, 0] == 7).all()
    only = pq.pq1_kv4_read(cache, slots.to(dev), k_out=wide[:, :, 0])
    assert only[1] is None and torch.equal(only[0].nan_to_num(0), k.nan_to_num(0))


def test_read4_of_every_byte(pq, dev):
    """All 256 code bytes under all 256 scales, in fp32."""
    cache = pq.KV4Cache.empty(256, 16, 1, 32, BF16, dev)
    codes = torch.arange(256, dtype=torch.uint8).view(16, 16).repeat(256, 1, 1).unsqueeze(1)
    scales = torch.arange(256, dtype=torch.uint8).view(256, 1, 1, 1).expand(256, 1, 16, 1)
    cache.k.copy_(codes)
    cache.k_scale.copy_(scales)
    out = torch.empty(4096, 1, 32, device=dev)
    pq.pq1_kv4_read(cache, torch.arange(4096, device=dev), k_out=out)
    want = ref4.values(codes, scales.contiguous()).transpose(1, 2).flatten(0, 1).to(F32)
    assert torch.equal(torch.isnan(out.cpu()), torch.isnan(want))
    assert torch.equal(out.cpu().nan_to_num(0), want.nan_to_num(0))


@pytest.mark.parametrize("dout", [BF16, F32], ids=["bf16", "f32"])
def test_read4_of_more_than_the_caches_hold(pq, dev, dout):
    """Outputs past 128 MB are stored another way: the same values, whole and in slices."""
    T, H, D = 70000, 4, 256
    cache = filled(pq, dev, 40, 64, H, D, BF16, 3)
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(100 + s % 50)
    slots = torch.randint(-3, 40 * 64 + 3, (T,), generator=torch.Generator().manual_seed(1)).to(dev)
    k, v = pq.pq1_kv4_read(cache, slots, out_dtype=dout)
    wide = torch.full((T, H, 2 * D), 7.0, dtype=dout, device=dev)
    pq.pq1_kv4_read(cache, slots, v_out=wide[:, :, D:])
    assert torch.equal(wide[:, :, D:], v) and bool((wide[:, :, :D] == 7).all())
    for at in (0, 30000, T - 1000):
        some = pq.pq1_kv4_read(cache, slots[at:at + 1000].contiguous(), out_dtype=dout)
        assert torch.equal(some[0], k[at:at + 1000]) and torch.equal(some[1], v[at:at + 1000])
    live = (slots >= 0) & (slots < 40 * 64)
    assert bool((k[~live] == 0).all()) and bool((v[~live] == 0).all())


def test_append4_and_read4_past_32_bits(pq, dev):
    """Rows more than 4 GB into the codes."""
    pages, page, H, D = 1 << 14, 64, 16, 512          # 2^24 rows of 256 bytes
    cache = pq.KV4Cache.empty(pages, page, H, D, BF16, dev)
    x = drawn((3, H, D), 1).to(dev)
    slots = torch.tensor([pages * page - 1, 5, (pages - 2) * page + 7], device=dev)
    pq.pq1_kv4_append(cache, x, -x, slots)
    k, v = pq.pq1_kv4_read(cache, slots, out_dtype=F32)
    want = ref4.quantise(x.cpu(), BF16)[0]
    assert torch.equal(k.double().cpu(), want) and torch.equal(v.double().cpu(), -want)


def test_calls_in_graphs_and_on_streams(pq, dev):
    """Append, read and the norm's gradient captured together, replayed on other data
    between eager calls; the gradient's workspace is the graph's own."""
    T, H, D = 70, 4, 128
    w = (1 + drawn((D,), 4, F32, 0.3)).to(dev)
    rope = pq.Rope(64, freqs=pq.rope_frequencies(64, device=dev))
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    norm = pq.HeadNorm(w, w, eps=1e-6)
    slots = torch.randperm(96, device=dev)[:T]

    def step(cache, x, g):
        q = pq.pq1_kv4_append(cache, x[:, :H], x[:, H:2 * H], slots, positions=pos, rope=rope,
                              q=x[:, 2 * H:], norm=norm)
        k, v = pq.pq1_kv4_read(cache, slots)
        return (q, k, v, *pq.pq1_norm_rope_grad(g, x[:, :H], w, pos, rope))

    make = lambda: pq.KV4Cache.empty(6, 16, H, D, BF16, dev)
    x, g = drawn((T, 3 * H, D), 1).to(dev), drawn((T, H, D), 2).to(dev)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    cache = make()
    with torch.cuda.stream(stream):
        step(cache, x, g)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = step(cache, x, g)
    torch.cuda.current_stream().wait_stream(stream)
    for seed in range(3, 8):
        x.copy_(drawn((T, 3 * H, D), seed))
        g.copy_(drawn((T, H, D), seed + 100))
        want = step(make(), x, g)
        graph.replay()
        step(make(), -x, -g)                    # eager work meanwhile
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_norm_past_32_bits(pq, dev):
    """More than 2^31 elements: the last tokens as in a call of their own, and the
    weight's gradient as that of two halves together."""
    T, H, D = 530000, 16, 256
    g = torch.Generator(device=dev).manual_seed(2)
    x = torch.randn(T, H, D, device=dev, dtype=BF16, generator=g)
    w = (1 + drawn((D,), 6, F32, 0.3)).to(dev)
    rope, _ = rotation(pq, dev, 64, (32,), "halves", False)
    pos = torch.arange(T, dtype=torch.int32, device=dev).flip(0)[None].contiguous()
    y = pq.pq1_norm_rope(x, w, pos, rope)
    for at in (0, T // 2 + 1, T - 7):
        few = slice(at, at + 7)
        assert torch.equal(y[few], pq.pq1_norm_rope(x[few].clone(), w, pos[:, few].contiguous(), rope))
    dx, _ = pq.pq1_norm_rope_grad(y, x, w, pos, rope, weight_grad=False)
    for at in (0, T - 7):
        few = slice(at, at + 7)
        assert torch.equal(dx[few], pq.pq1_norm_rope_grad(y[few].clone(), x[few].clone(), w,
                                                          pos[:, few].contiguous(), rope,
                                                          weight_grad=False)[0])
    # a workgroup's lanes add up at most T H / 1024 heads in fp32, every eighth each
    # and then their eight sums; what is added is off by a few 2^-24 of itself
    half = T // 2
    _, dw = pq.pq1_norm_rope_grad(y, x, w, dx=dx)
    parts = [pq.pq1_norm_rope_grad(y[c], x[c], w, dx=dx[c])[1].double()
             for c in (slice(0, half), slice(half, T))]
    _, size = pq.pq1_norm_rope_grad(y.abs_(), x.abs_(), w, dx=dx)
    bound = 2 * (T * H / 1024 / 8 + 8 + 8) * 2.0 ** -24 * size.double()
    assert bool(((dw.double() - parts[0] - parts[1]).abs() <= bound).all())
