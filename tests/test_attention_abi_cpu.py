"""The attention-layer calls without a GPU: what they refuse (before the HIP
runtime is touched), what the binding refuses, and the 64-bit forms that the
GPU tests rest on."""
import ctypes
import math

import pytest
import torch
from hypothesis import HealthCheck, given, settings, strategies as st

import attention_reference as ref
from conftest import gpu_available
from gemm_hadamard_rotated_amd import pq1

needs_no_gpu = pytest.mark.skipif(gpu_available(), reason="needs a host without a visible GPU")

OK, NULL, SHAPE, ALIGN, ALIAS, ARG = 0, 1, 2, 3, 5, 8
F32, BF16, GEMM, F16 = 0, 1, 2, 3
P = ctypes.c_void_p
GIB = 1 << 30
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(pq1.LIB_PATH):
        from gemm_hadamard_rotated_amd import build
        build.build()
    return pq1.load_library()


def heads(at, dtype=BF16, ts=None, hs=128, n=8, D=128):
    """A made-up view, never dereferenced."""
    return pq1.Pq1Heads(at, dtype, n * D if ts is None else ts, hs)


def spec(rot=64, axes=1, section=(32, 0, 0, 0), interleaved=0, pairing=0, inverse=0):
    return pq1.Pq1RopeSpec(rot, axes, (ctypes.c_int32 * 4)(*section), interleaved, pairing, inverse)


def cache(k=BIG, v=2 * BIG, dtype=BF16, page=16, pages=64, n=8, D=128):
    return pq1.Pq1KvCache(k, v, dtype, page, pages, n, D)


# ---------------------------------------------------------------------------
# Rotation
# ---------------------------------------------------------------------------
def rope(lib, x=None, y=None, pos=P(3 * GIB), fr=P(4 * GIB), s=None, T=4, H=8, D=128):
    return lib.pq1_rope(heads(GIB) if x is None else x, heads(2 * GIB) if y is None else y, pos, fr,
                        spec() if s is None else s, T, H, D, None)


def test_rope_refusals(lib):
    r = lambda **kw: rope(lib, **kw)
    assert lib.pq1_rope(None, heads(GIB), P(8), P(8), spec(), 4, 8, 128, None) == NULL
    assert lib.pq1_rope(heads(GIB), None, P(8), P(8), spec(), 4, 8, 128, None) == NULL
    assert lib.pq1_rope(heads(GIB), heads(GIB), P(8), P(8), None, 4, 8, 128, None) == NULL
    assert r(x=heads(None)) == NULL and r(y=heads(None)) == NULL
    assert r(pos=None) == NULL and r(fr=None) == NULL
    assert r(x=heads(GIB, GEMM)) == ARG and r(y=heads(GIB, 4)) == ARG and r(x=heads(GIB, -1)) == ARG
    for T, H, D in ((-1, 8, 128), (4, 0, 128), (4, -1, 128), (4, 1025, 128), (4, 8, 0), (4, 8, 12),
                    (4, 8, 1032), (1 << 30, 8, 128), (1 << 29, 1024, 1024)):
        assert r(T=T, H=H, D=D) == SHAPE, (T, H, D)
    for s in (spec(rot=0), spec(rot=63), spec(rot=130, section=(65, 0, 0, 0)), spec(axes=0),
              spec(axes=5), spec(section=(31, 0, 0, 0)), spec(section=(33, 0, 0, 0)),
              spec(axes=2, section=(-1, 33, 0, 0)), spec(axes=2, section=(10, 10, 0, 0)),
              # interleaved: the second axis would need a pair past the last
              spec(axes=2, section=(10, 22, 0, 0), interleaved=1)):
        assert r(s=s) == SHAPE
    assert r(s=spec(interleaved=2)) == ARG
    assert r(s=spec(pairing=2)) == ARG and r(s=spec(pairing=-1)) == ARG
    assert r(s=spec(inverse=-1)) == ARG
    assert r(x=heads(GIB + 8)) == ALIGN and r(y=heads(GIB + 2)) == ALIGN
    assert r(x=heads(GIB, ts=1028)) == ALIGN and r(x=heads(GIB, hs=4)) == ALIGN
    assert r(pos=P(GIB + 2)) == ALIGN and r(fr=P(GIB + 4)) == ALIGN
    assert r(x=heads(GIB, ts=-1024)) == SHAPE and r(x=heads(GIB, hs=-128)) == SHAPE
    assert r(x=heads(GIB, ts=(1 << 31) + 8)) == SHAPE
    # outputs over inputs, and over themselves
    assert r(y=heads(GIB + 1024)) == ALIAS
    assert r(y=heads(GIB, F32)) == ALIAS                    # in place needs the same type
    assert r(x=heads(GIB, ts=2048), y=heads(GIB)) == ALIAS  # and strides
    assert r(pos=P(2 * GIB + 64)) == ALIAS and r(fr=P(2 * GIB + 64)) == ALIAS
    assert r(y=heads(2 * GIB, ts=512)) == ALIAS             # tokens run into one another
    assert r(y=heads(2 * GIB, hs=0)) == ALIAS
    assert r(T=0) == OK and r(T=0, x=heads(None), pos=None) == OK


@needs_no_gpu
def test_rope_accepted_up_to_the_device_check(lib):
    ok = {6}
    assert rope(lib) in ok and rope(lib, y=heads(GIB)) in ok      # in place
    assert rope(lib, x=heads(GIB, F32), y=heads(2 * GIB, F16), T=1) in ok
    # the strides of single tokens and heads may be anything
    assert rope(lib, x=heads(GIB, ts=0, hs=0), y=heads(2 * GIB, ts=0, hs=0), T=1, H=1) in ok
    assert rope(lib, y=heads(2 * GIB, ts=128, hs=512), T=4) in ok   # heads outside tokens
    assert rope(lib, s=spec(axes=3, section=(11, 11, 10, 0), interleaved=1)) in ok
    assert rope(lib, s=spec(axes=4, section=(8, 8, 8, 8), pairing=1, inverse=1)) in ok


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
def append(lib, k=None, v=None, slots=P(3 * GIB), q=None, qo=None, Hq=16, pos=P(4 * GIB),
           fr=P(5 * GIB), s=None, c=None, T=4):
    return lib.pq1_kv_append(heads(GIB) if k is None else k, heads(2 * GIB) if v is None else v,
                             slots, q, qo, Hq, pos, fr, s, cache() if c is None else c, T, None)


def test_append_refusals(lib):
    a = lambda **kw: append(lib, **kw)
    q, qo = heads(6 * GIB, n=16), heads(7 * GIB, n=16)
    assert lib.pq1_kv_append(None, heads(GIB), P(8), None, None, 0, None, None, None, cache(), 4,
                             None) == NULL
    assert lib.pq1_kv_append(heads(GIB), heads(GIB), P(8), None, None, 0, None, None, None, None,
                             4, None) == NULL
    assert a(slots=None) == NULL and a(q=q) == NULL and a(q=heads(None), qo=qo) == NULL
    assert a(s=spec(), pos=None) == NULL and a(s=spec(), fr=None) == NULL
    assert a(c=cache(k=None)) == NULL and a(c=cache(v=None)) == NULL
    assert a(k=heads(GIB, F16)) == ARG                      # neither fp32 nor the cache's type
    assert a(v=heads(2 * GIB, F32)) == ARG                  # not k's
    assert a(q=heads(6 * GIB, F32, n=16), qo=qo) == ARG
    assert a(q=q, qo=heads(7 * GIB, F32, n=16)) == ARG
    assert a(c=cache(dtype=F32)) == ARG and a(s=spec(pairing=7)) == ARG
    for c in (cache(pages=0), cache(n=0), cache(n=1025), cache(D=12), cache(D=0), cache(D=1032),
              cache(page=0), cache(page=24), cache(page=1 << 17), cache(page=-16),
              cache(pages=1 << 31), cache(pages=1 << 30, page=65536)):
        assert a(c=c) == SHAPE
    assert a(q=q, qo=qo, Hq=0) == SHAPE and a(q=q, qo=qo, Hq=1025) == SHAPE
    assert a(T=-1) == SHAPE and a(T=1 << 30) == SHAPE
    assert a(s=spec(rot=130, section=(65, 0, 0, 0))) == SHAPE
    assert a(k=heads(GIB + 8)) == ALIGN and a(v=heads(2 * GIB, ts=1028)) == ALIGN
    assert a(slots=P(GIB + 4)) == ALIGN and a(c=cache(k=BIG + 8)) == ALIGN
    assert a(q=q, qo=heads(7 * GIB + 8, n=16)) == ALIGN
    assert a(s=spec(), pos=P(GIB + 1)) == ALIGN
    assert a(k=heads(BIG + 4096)) == ALIAS and a(v=heads(2 * BIG)) == ALIAS
    assert a(slots=P(BIG)) == ALIAS and a(c=cache(v=BIG + 4096)) == ALIAS
    assert a(q=q, qo=heads(6 * GIB, n=16)) == ALIAS and a(q=q, qo=heads(BIG, n=16)) == ALIAS
    assert a(q=q, qo=heads(7 * GIB, ts=1024)) == ALIAS      # 16 heads do not fit 1024 elements
    assert a(s=spec(), pos=P(BIG)) == ALIAS and a(s=spec(), fr=P(2 * BIG + 64)) == ALIAS
    assert a(T=0) == OK and a(T=0, slots=None) == OK


@needs_no_gpu
def test_append_accepted_up_to_the_device_check(lib):
    q, qo = heads(6 * GIB, n=16), heads(7 * GIB, n=16)
    assert append(lib) == 6                                  # Hq is ignored without q
    assert append(lib, Hq=-5, pos=None, fr=None) == 6
    assert append(lib, q=q, qo=qo, s=spec()) == 6
    assert append(lib, k=heads(GIB), v=heads(GIB)) == 6      # inputs may overlap
    assert append(lib, k=heads(GIB, F32), v=heads(2 * GIB, F32), c=cache(dtype=F16)) == 6


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
def attend(lib, q=None, out=None, c=None, table=P(3 * GIB), max_pages=10, cu=P(4 * GIB),
           kv=P(5 * GIB), B=2, T=4, Hq=16, max_q=2, max_kv=160, scale=0.1, causal=1, window=0,
           ws=P(8 * GIB), wsb=1 << 28):
    return lib.pq1_paged_attention(heads(GIB, n=16) if q is None else q,
                                   heads(2 * GIB, n=16) if out is None else out,
                                   cache() if c is None else c, table, max_pages, cu, kv, B, T, Hq,
                                   max_q, max_kv, scale, causal, window, ws, wsb, None)


def test_attention_refusals(lib):
    a = lambda **kw: attend(lib, **kw)
    assert lib.pq1_paged_attention(None, heads(GIB), cache(), P(8), 1, P(8), P(8), 1, 1, 8, 1, 1,
                                   0.1, 1, 0, None, 0, None) == NULL
    assert a(q=heads(None)) == NULL and a(out=heads(None)) == NULL
    assert a(table=None) == NULL and a(cu=None) == NULL and a(kv=None) == NULL
    assert a(c=cache(k=None)) == NULL
    assert a(q=heads(GIB, F16, n=16)) == ARG and a(out=heads(2 * GIB, F16, n=16)) == ARG
    assert a(q=heads(GIB, F32, n=16)) == ARG and a(c=cache(dtype=F32)) == ARG
    for scale in (0.0, -1.0, math.inf, -math.inf, math.nan, 3e38):
        assert a(scale=scale) == ARG, scale
    assert a(causal=2) == ARG and a(causal=-1) == ARG and a(window=-1) == ARG
    assert a(causal=0, window=5) == ARG
    for kw in (dict(Hq=15), dict(Hq=4), dict(Hq=0), dict(Hq=1032), dict(B=-1), dict(T=-1),
               dict(max_q=-1), dict(max_kv=-1), dict(max_pages=-1), dict(max_pages=1 << 31),
               dict(T=1 << 30), dict(T=1 << 28), dict(B=1 << 30), dict(B=1 << 24),
               dict(c=cache(D=80)), dict(c=cache(D=512)), dict(c=cache(page=48)),
               dict(c=cache(pages=0))):
        assert a(**kw) == SHAPE, kw
    assert a(q=heads(GIB + 4, n=16)) == ALIGN and a(out=heads(2 * GIB, ts=2052)) == ALIGN
    assert a(table=P(GIB + 2)) == ALIGN and a(cu=P(GIB + 1)) == ALIGN and a(kv=P(GIB + 3)) == ALIGN
    assert a(out=heads(GIB, n=16)) == ALIAS and a(out=heads(BIG, n=16)) == ALIAS
    assert a(out=heads(3 * GIB - 64, n=16)) == ALIAS        # the table
    assert a(out=heads(4 * GIB, n=16)) == ALIAS and a(out=heads(5 * GIB, n=16)) == ALIAS
    assert a(out=heads(2 * GIB, ts=1024)) == ALIAS and a(out=heads(2 * GIB, hs=64)) == ALIAS
    # a workspace is needed where the keys are cut into parts
    far = dict(max_kv=100000, max_pages=10000)
    need = lib.pq1_paged_attention_workspace_bytes(2, 4, 16, 8, 128, 2, 100000)
    assert need > 0
    assert a(ws=None, **far) == NULL and a(ws=P(8 * GIB + 128), **far) == ALIGN
    assert a(wsb=need - 1, **far) == ARG
    assert a(ws=P(GIB), **far) == ALIAS and a(ws=P(2 * GIB), **far) == ALIAS
    assert a(B=0) == OK and a(T=0) == OK and a(B=0, cu=None, q=heads(None)) == OK


@needs_no_gpu
def test_attention_accepted_up_to_the_device_check(lib):
    assert attend(lib) == 6
    assert attend(lib, ws=None, wsb=0) == 6                  # a short cache needs no workspace
    assert attend(lib, table=None, max_pages=0) == 6
    assert attend(lib, out=heads(2 * GIB, F32, n=16), causal=0) == 6
    assert attend(lib, window=1 << 30, max_kv=1 << 62) == 6
    need = lib.pq1_paged_attention_workspace_bytes(2, 4, 16, 8, 128, 2, 100000)
    assert attend(lib, max_kv=100000, wsb=need) == 6


def test_attention_workspace_bytes(lib):
    f = lib.pq1_paged_attention_workspace_bytes
    for bad in ((2, 4, 15, 8, 128, 2, 9), (2, 4, 16, 8, 80, 2, 9), (-1, 4, 16, 8, 128, 2, 9),
                (2, 4, 16, 0, 128, 2, 9), (2, 1 << 30, 16, 8, 128, 2, 9), (0, 4, 16, 8, 128, 2, 9),
                (2, 0, 16, 8, 128, 2, 9)):
        assert f(*bad) == 0
    for B, T, Hq, H, D, mq, mkv in ((1, 1, 24, 4, 256, 1, 131071), (64, 64, 24, 4, 256, 1, 8000),
                                    (16, 96, 32, 8, 128, 6, 4000), (1, 2048, 24, 4, 256, 2048, 8192),
                                    (1, 100, 8, 1, 64, 100, 1 << 31)):
        n = f(B, T, Hq, H, D, mq, mkv)
        row = T * Hq * (4 * D + 8)
        assert n % row == 0 and n <= 512 * row
        # no less for a longer cache
        assert f(B, T, Hq, H, D, mq, 2 * mkv) >= n


ptr = st.one_of(st.just(None), st.builds(lambda k, off: (1 << 36) * k + off, st.integers(1, 8),
                                         st.sampled_from([0, 0, 0, 2, 4, 8, 256])))
size = st.one_of(st.sampled_from([-1, 0, 1, 7, 64, 1000, 1 << 20, (1 << 31) - 1, 1 << 31, 1 << 40,
                                  (1 << 63) - 1, -(1 << 63)]), st.integers(-5, 5000))
small = st.one_of(st.sampled_from([-1, 0, 1, 2, 4, 8, 24, 64, 128, 256, 1024, (1 << 31) - 1,
                                   -(1 << 31)]), st.integers(-3, 40))
view = st.builds(pq1.Pq1Heads, ptr, st.integers(-1, 4), size, size)
spec_any = st.builds(lambda r, a, s, i, p, v: spec(r, a, s, i, p, v), small, st.integers(-1, 5),
                     st.tuples(small, small, small, small), st.integers(-1, 2),
                     st.integers(-1, 2), st.integers(-1, 2))
cache_any = st.builds(pq1.Pq1KvCache, ptr, ptr, st.integers(-1, 4), small, size, small, small)
opt = lambda s: st.one_of(st.none(), s)
SETTINGS = dict(max_examples=400, deadline=None, derandomize=True,
                suppress_health_check=[HealthCheck.function_scoped_fixture])
CODES = {0, 1, 2, 3, 5, 6, 8}


@needs_no_gpu
@settings(**SETTINGS)
@given(x=opt(view), y=opt(view), p=ptr, f=ptr, s=opt(spec_any), T=size, H=small, D=small)
def test_rope_any_arguments(lib, x, y, p, f, s, T, H, D):
    assert lib.pq1_rope(x, y, p, f, s, T, H, D, None) in CODES


@needs_no_gpu
@settings(**SETTINGS)
@given(k=opt(view), v=opt(view), sl=ptr, q=opt(view), qo=opt(view), Hq=small, p=ptr, f=ptr,
       s=opt(spec_any), c=opt(cache_any), T=size)
def test_append_any_arguments(lib, k, v, sl, q, qo, Hq, p, f, s, c, T):
    assert lib.pq1_kv_append(k, v, sl, q, qo, Hq, p, f, s, c, T, None) in CODES


@needs_no_gpu
@settings(**SETTINGS)
@given(q=opt(view), o=opt(view), c=opt(cache_any), t=ptr, mp=size, cu=ptr, kv=ptr, B=size, T=size,
       Hq=small, mq=size, mkv=size, sc=st.floats(width=32), ca=st.integers(-1, 2), w=small, ws=ptr,
       wsb=st.sampled_from([0, 1 << 20, 1 << 40]))
def test_attention_any_arguments(lib, q, o, c, t, mp, cu, kv, B, T, Hq, mq, mkv, sc, ca, w, ws,
                                 wsb):
    assert lib.pq1_paged_attention(q, o, c, t, mp, cu, kv, B, T, Hq, mq, mkv, sc, ca, w, ws, wsb,
                                   None) in CODES
    H, D = (c.heads, c.dim) if c is not None else (4, 64)
    assert lib.pq1_paged_attention_workspace_bytes(B, T, Hq, H, D, mq, mkv) >= 0


@needs_no_gpu
@settings(**SETTINGS)
@given(B=st.integers(1, 1 << 23), T=st.integers(1, 1 << 30), Hk=st.integers(1, 1024),
       G=st.integers(1, 64), D=st.sampled_from([64, 128, 256]), mq=st.integers(0, 1 << 62),
       mkv=st.integers(0, 1 << 62), w=st.integers(0, (1 << 31) - 1))
def test_attention_plans_of_any_size(lib, B, T, Hk, G, D, mq, mkv, w):
    """Sizes alone: a plan is refused, or the workspace it asked for does."""
    c = cache(n=Hk, D=D, k=1 << 50, v=1 << 51)
    need = lib.pq1_paged_attention_workspace_bytes(B, T, Hk * G, Hk, D, mq, mkv)
    got = attend(lib, c=c, q=heads(1 << 52, n=Hk * G, D=D, hs=D),
                 out=heads(1 << 53, n=Hk * G, D=D, hs=D), table=P(1 << 54), cu=P(1 << 55),
                 kv=P(1 << 56), B=B, T=T, Hq=Hk * G, max_q=mq, max_kv=mkv, window=w,
                 ws=P(1 << 57), wsb=need)
    assert got in (SHAPE, 6)


# ---------------------------------------------------------------------------
# Binding
# ---------------------------------------------------------------------------
def test_binding_refuses_cpu_tensors_and_other_types():
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        pq1.Rope(32, freqs=pq1.rope_frequencies(32))
    with pytest.raises(ValueError, match="GPU"):
        pq1.KVCache(x, x) if x.dtype == torch.bfloat16 else pq1.KVCache(
            torch.zeros(1, 1, 1, 8, dtype=torch.bfloat16), torch.zeros(1, 1, 1, 8))
    with pytest.raises(ValueError, match="GPU"):
        pq1.pq1_rope(x, torch.zeros(1, 2, dtype=torch.int32), None)
    with pytest.raises(TypeError, match="KVCache"):
        pq1.pq1_kv_append(None, x, x, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(TypeError, match="KVCache"):
        pq1.pq1_paged_attention(x, None, x, x, x, 1, 1)


def test_no_other_call_lost_its_error_check():
    """Every failing call raises with its own name."""
    with pytest.raises(pq1.Pq1Error, match="pq1_gemv"):
        pq1._check(SHAPE, "pq1_gemv")


# ---------------------------------------------------------------------------
# The 64-bit forms themselves
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
@pytest.mark.parametrize("sections,interleaved", [((8,), False), ((3, 3, 2), True),
                                                  ((2, 6), False), ((0, 8), False)])
def test_reference_rotation(pairing, sections, interleaved):
    T, H, D, rot = 6, 2, 24, 16
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, D, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 50, (len(sections), T), generator=g)
    f = pq1.rope_frequencies(rot, 100.0)
    assert abs(float(f[3]) - 100.0 ** (-6 / 16)) < 1e-15
    y, _ = ref.rotate(x, pos, f, sections, pairing, interleaved)
    owner = ref.axis_of_pair(rot, sections, interleaved)
    assert [owner.count(a) for a in range(len(sections))] == list(sections)
    for t in range(T):
        for i in range(rot // 2):
            a, b = (i, i + rot // 2) if pairing == "halves" else (2 * i, 2 * i + 1)
            th = float(pos[owner[i], t]) * float(f[i])
            z = (x[t, :, a] + 1j * x[t, :, b]) * complex(math.cos(th), math.sin(th))
            assert torch.allclose(y[t, :, a], z.real, atol=1e-12)
            assert torch.allclose(y[t, :, b], z.imag, atol=1e-12)
    back, _ = ref.rotate(y, pos, f, sections, pairing, interleaved, inverse=True)
    assert torch.allclose(back, x, atol=1e-12) and torch.equal(y[..., rot:], x[..., rot:])


def test_reference_attention():
    g = torch.Generator().manual_seed(2)
    q = torch.randn(3, 4, 8, generator=g)
    k, v = torch.randn(7, 2, 8, generator=g), torch.randn(7, 2, 8, generator=g)
    o, w, _ = ref.attention(q, k, v, 0.5, True, 4)
    for i in range(3):
        p = 7 - 3 + i
        for h in range(4):
            e = [math.exp(0.5 * float(q[i, h].double() @ k[j, h // 2].double()))
                 for j in range(p - 3, p + 1)]
            want = sum(a * v[j, h // 2].double() for a, j in zip(e, range(p - 3, p + 1))) / sum(e)
            assert torch.allclose(o[i, h], want, atol=1e-12)
    assert bool((w >= o.abs() - 1e-12).all())
    o, _, _ = ref.attention(q, k[:2], v[:2], 0.5, True, 0)      # the first row sees no key
    assert bool((o[0] == 0).all()) and not bool((o[1] == 0).any())
