"""The calls around per-head norms and 4-bit caches without a GPU: what they
refuse (before the HIP runtime is touched), and what the binding refuses."""
import ctypes
import math

import pytest
import torch
from hypothesis import given, settings, strategies as st

import kv4_reference as ref4
from conftest import gpu_available
from gemm_hadamard_rotated_amd import pq1
from test_attention_abi_cpu import (ALIAS, ALIGN, ARG, BF16, BIG, CODES, F16, F32, GEMM, GIB, NULL,
                                    OK, P, SETTINGS, SHAPE, cache, cache_any, heads, lib, opt,  # noqa: F401
                                    ptr, size, small, spec, spec_any, view)

needs_no_gpu = pytest.mark.skipif(gpu_available(), reason="needs a host without a visible GPU")
DEVICE = 6


def norm(lib, x=None, y=None, w=P(5 * GIB), eps=1e-6, pos=P(3 * GIB), fr=P(4 * GIB), s="spec", T=4, H=8,
         D=128):
    return lib.pq1_norm_rope(heads(GIB) if x is None else x, heads(2 * GIB) if y is None else y, w,
                             eps, pos, fr, spec() if s == "spec" else s, T, H, D, None)


def test_norm_refusals(lib):  # noqa: F811
    r = lambda **kw: norm(lib, **kw)
    assert lib.pq1_norm_rope(None, heads(GIB), P(8), 1.0, None, None, None, 4, 8, 128, None) == NULL
    assert lib.pq1_norm_rope(heads(GIB), None, P(8), 1.0, None, None, None, 4, 8, 128, None) == NULL
    assert r(x=heads(None)) == NULL and r(y=heads(None)) == NULL and r(w=None) == NULL
    assert r(pos=None) == NULL and r(fr=None) == NULL
    for eps in (0.0, -1.0, math.inf, math.nan, 1e-60):
        assert r(eps=eps) == ARG
    assert r(x=heads(GIB, GEMM)) == ARG and r(y=heads(GIB, 4)) == ARG
    for T, H, D in ((-1, 8, 128), (4, 0, 128), (4, 1025, 128), (4, 8, 0), (4, 8, 12), (4, 8, 1032),
                    (1 << 30, 8, 128), (1 << 29, 1024, 1024)):
        assert r(T=T, H=H, D=D) == SHAPE
        assert r(T=T, H=H, D=D, s=None) == SHAPE
    assert r(s=spec(rot=63)) == SHAPE and r(s=spec(interleaved=2)) == ARG
    assert r(w=P(5 * GIB + 4)) == ALIGN and r(x=heads(GIB + 8)) == ALIGN
    assert r(pos=P(GIB + 2)) == ALIGN and r(fr=P(GIB + 4)) == ALIGN
    assert r(y=heads(GIB + 1024)) == ALIAS and r(w=P(2 * GIB + 64)) == ALIAS
    assert r(pos=P(2 * GIB + 64)) == ALIAS and r(fr=P(2 * GIB + 64)) == ALIAS
    assert r(y=heads(2 * GIB, ts=512)) == ALIAS
    assert r(T=0) == OK and r(T=0, x=heads(None), w=None) == OK


@needs_no_gpu
def test_norm_accepted_up_to_the_device_check(lib):  # noqa: F811
    assert norm(lib) == DEVICE and norm(lib, y=heads(GIB)) == DEVICE
    assert norm(lib, s=None, pos=None, fr=None) == DEVICE
    assert norm(lib, x=heads(GIB, F32), y=heads(2 * GIB, F16), T=1, eps=2.0 ** -149) == DEVICE


def grad(lib, g=None, x=None, dx=None, w=P(5 * GIB), dw=P(6 * GIB), eps=1e-6, pos=P(3 * GIB),
         fr=P(4 * GIB), s="spec", T=4, H=8, D=128, ws=P(7 * GIB), n=1 << 20):
    return lib.pq1_norm_rope_grad(heads(GIB) if g is None else g, heads(2 * GIB) if x is None else x,
                                  heads(8 * GIB) if dx is None else dx, w, dw, eps, pos, fr,
                                  spec() if s == "spec" else s, T, H, D, ws, n, None)


def test_norm_grad_refusals(lib):  # noqa: F811
    r = lambda **kw: grad(lib, **kw)
    for i in range(3):
        views = [heads((i + 1) * GIB) for i in range(3)]
        views[i] = None
        assert lib.pq1_norm_rope_grad(*views, P(8), None, 1.0, None, None, None, 4, 8, 128, None, 0,
                                      None) == NULL
    assert r(g=heads(None)) == NULL and r(x=heads(None)) == NULL and r(dx=heads(None)) == NULL
    assert r(w=None) == NULL and r(pos=None) == NULL and r(ws=None) == NULL
    assert r(g=heads(GIB, GEMM)) == ARG and r(x=heads(GIB, 9)) == ARG
    assert r(dx=heads(8 * GIB, F32)) == ARG and r(eps=0.0) == ARG
    assert lib.pq1_norm_rope_grad_workspace_bytes(4, 128) == 4 * 128 * 4
    assert r(n=4 * 128 * 4 - 1) == ARG
    assert r(T=-1) == SHAPE and r(H=0) == SHAPE and r(D=4) == SHAPE and r(s=spec(rot=130)) == SHAPE
    assert r(dw=P(6 * GIB + 2)) == ALIGN and r(ws=P(7 * GIB + 64)) == ALIGN
    assert r(w=P(5 * GIB + 8)) == ALIGN and r(dx=heads(8 * GIB + 8)) == ALIGN
    assert r(dx=heads(GIB + 1024)) == ALIAS and r(dx=heads(2 * GIB + 1024)) == ALIAS
    assert r(dx=heads(8 * GIB, ts=512)) == ALIAS
    for at in (GIB, 2 * GIB, 3 * GIB, 4 * GIB, 5 * GIB, 8 * GIB):
        assert r(dw=P(at)) == ALIAS and r(ws=P(at)) == ALIAS
    assert r(dw=P(7 * GIB)) == ALIAS
    for T, D in ((-1, 128), (4, 12), (4, 1032), (1 << 30, 128)):
        assert lib.pq1_norm_rope_grad_workspace_bytes(T, D) == 0
    assert lib.pq1_norm_rope_grad_workspace_bytes(1 << 29, 128) == 1024 * 128 * 4
    assert r(T=0, dw=None) == OK


@needs_no_gpu
def test_norm_grad_accepted_up_to_the_device_check(lib):  # noqa: F811
    assert grad(lib) == DEVICE and grad(lib, dw=None, ws=None, n=0) == DEVICE
    assert grad(lib, dx=heads(GIB)) == DEVICE and grad(lib, dx=heads(2 * GIB)) == DEVICE
    assert grad(lib, T=0, ws=None, n=0) == DEVICE      # dweight becomes zeros


def cache4(k=BIG, ks=2 * BIG, v=3 * BIG, vs=4 * BIG, dtype=BF16, page=16, pages=64, n=8, D=128):
    return pq1.Pq1Kv4Cache(k, ks, v, vs, dtype, page, pages, n, D)


def hnorm(q=9 * GIB, k=10 * GIB, eps=1e-6):
    return pq1.Pq1HeadNorm(q, k, eps)


def append4(lib, k=None, v=None, slots=P(3 * GIB), q=None, qo=None, Hq=16, pos=P(4 * GIB),
            fr=P(5 * GIB), s=None, nm=None, c=None, T=4, fn="pq1_kv4_append"):
    c = (cache4() if fn == "pq1_kv4_append" else cache()) if c is None else c
    return getattr(lib, fn)(heads(GIB) if k is None else k, heads(2 * GIB) if v is None else v, slots,
                            q, qo, Hq, pos, fr, s, nm, c, T, None)


@pytest.mark.parametrize("fn", ["pq1_kv4_append", "pq1_kv_append_ex"])
def test_append_refusals(lib, fn):  # noqa: F811
    nm = hnorm()
    a = lambda **kw: append4(lib, **{"fn": fn, "nm": nm, **kw})
    make = cache4 if fn == "pq1_kv4_append" else cache
    q, qo = heads(6 * GIB, n=16), heads(7 * GIB, n=16)
    call = getattr(lib, fn)
    assert call(None, heads(GIB), P(8), None, None, 0, None, None, None, nm, make(), 4, None) == NULL
    assert call(heads(GIB), None, P(8), None, None, 0, None, None, None, nm, make(), 4, None) == NULL
    assert call(heads(GIB), heads(GIB), P(8), None, None, 0, None, None, None, nm, None, 4, None) == NULL
    assert a(slots=None) == NULL and a(q=q) == NULL and a(q=heads(None), qo=qo) == NULL
    assert a(s=spec(), pos=None) == NULL and a(s=spec(), fr=None) == NULL
    assert a(c=make(k=None)) == NULL and a(c=make(v=None)) == NULL
    assert a(k=heads(GIB, F16)) == ARG and a(v=heads(2 * GIB, F32)) == ARG
    assert a(q=heads(6 * GIB, F32, n=16), qo=qo) == ARG and a(q=q, qo=heads(7 * GIB, F32, n=16)) == ARG
    assert a(c=make(dtype=F32)) == ARG and a(nm=hnorm(eps=0.0)) == ARG and a(nm=hnorm(eps=math.nan)) == ARG
    assert a(s=spec(interleaved=3)) == ARG
    for bad in (dict(page=0), dict(page=3), dict(page=1 << 17), dict(pages=0), dict(pages=1 << 31),
                dict(n=0), dict(n=1025), dict(D=0), dict(D=1032), dict(pages=1 << 30, page=65536)):
        assert a(c=make(**bad)) == SHAPE, bad
    assert a(q=q, qo=qo, Hq=0) == SHAPE and a(q=q, qo=qo, Hq=1025) == SHAPE
    assert a(T=-1) == SHAPE and a(T=1 << 30) == SHAPE and a(s=spec(rot=130, section=(65, 0, 0, 0))) == SHAPE
    assert a(slots=P(3 * GIB + 4)) == ALIGN and a(k=heads(GIB + 8)) == ALIGN
    assert a(c=make(k=BIG + 8)) == ALIGN and a(s=spec(), fr=P(5 * GIB + 4)) == ALIGN
    assert a(nm=hnorm(k=10 * GIB + 4)) == ALIGN and a(nm=hnorm(q=9 * GIB + 8), q=q, qo=qo) == ALIGN
    # outputs over inputs, and over one another
    for at in (GIB, 2 * GIB, 3 * GIB, 10 * GIB):
        assert a(c=make(k=at)) == ALIAS and a(c=make(v=at)) == ALIAS
        assert a(q=q, qo=heads(at, n=16)) == ALIAS
    assert a(c=make(v=BIG + 1024)) == ALIAS and a(q=q, qo=q) == ALIAS
    assert a(q=q, qo=heads(BIG, n=16)) == ALIAS and a(q=q, qo=heads(7 * GIB, ts=0, n=16)) == ALIAS
    assert a(s=spec(), c=make(k=4 * GIB)) == ALIAS and a(s=spec(), c=make(k=5 * GIB)) == ALIAS
    assert a(T=0) == OK and a(T=0, slots=None) == OK


def test_append4_refusals_of_its_cache(lib):  # noqa: F811
    a = lambda **kw: append4(lib, c=cache4(**kw))
    assert a(ks=None) == NULL and a(vs=None) == NULL
    assert a(ks=2 * BIG + 8) == ALIGN and a(vs=4 * BIG + 1) == ALIGN
    assert a(D=136) == SHAPE and a(D=16) == SHAPE
    for at in (GIB, 2 * GIB, 3 * GIB, BIG, 3 * BIG):
        assert a(ks=at) == ALIAS and a(vs=at) == ALIAS
    assert a(ks=4 * BIG) == ALIAS


@needs_no_gpu
def test_append4_accepted_up_to_the_device_check(lib):  # noqa: F811
    q, qo = heads(6 * GIB, n=16), heads(7 * GIB, n=16)
    for nm in (None, hnorm(), hnorm(q=None), hnorm(k=None), hnorm(q=None, k=None)):
        assert append4(lib, nm=nm) == DEVICE and append4(lib, nm=nm, q=q, qo=qo, s=spec()) == DEVICE
        assert append4(lib, nm=nm, fn="pq1_kv_append_ex") == DEVICE
    # a weight of queries that are not there is not looked at
    assert append4(lib, nm=hnorm(q=3)) == DEVICE
    assert append4(lib, k=heads(GIB, F32), v=heads(2 * GIB, F32), c=cache4(dtype=F16)) == DEVICE


def read4(lib, c="cache", slots=P(3 * GIB), k="view", v="view", T=4):
    return lib.pq1_kv4_read(cache4() if c == "cache" else c, slots, heads(GIB) if k == "view" else k,
                            heads(2 * GIB) if v == "view" else v, T, None)


def test_read4_refusals(lib):  # noqa: F811
    r = lambda **kw: read4(lib, **kw)
    assert r(c=None) == NULL and r(k=None, v=None) == NULL and r(slots=None) == NULL
    assert r(k=heads(None)) == NULL and r(v=heads(None)) == NULL and r(c=cache4(ks=None)) == NULL
    assert r(k=heads(GIB, F32)) == ARG and r(k=heads(GIB, GEMM), v=None) == ARG
    assert r(c=cache4(dtype=F32)) == ARG
    assert r(T=-1) == SHAPE and r(T=1 << 30) == SHAPE and r(c=cache4(D=72)) == SHAPE
    assert r(slots=P(3 * GIB + 4)) == ALIGN and r(v=heads(2 * GIB + 8)) == ALIGN
    assert r(k=heads(2 * GIB)) == ALIAS and r(k=heads(3 * GIB)) == ALIAS
    for at in (BIG, 2 * BIG, 3 * BIG, 4 * BIG):
        assert r(v=heads(at)) == ALIAS
    assert r(v=heads(2 * GIB, ts=512)) == ALIAS
    assert r(T=0) == OK and r(T=0, slots=None) == OK


@needs_no_gpu
def test_read4_accepted_up_to_the_device_check(lib):  # noqa: F811
    assert read4(lib) == DEVICE and read4(lib, k=None) == DEVICE and read4(lib, v=None) == DEVICE
    assert read4(lib, k=heads(GIB, F32), v=heads(2 * GIB, F32)) == DEVICE


# ---------------------------------------------------------------------------
# The binding
# ---------------------------------------------------------------------------
def test_binding_refuses_what_is_not_on_a_gpu():
    x = torch.zeros(4, 2, 64)
    with pytest.raises(ValueError, match="GPU"):
        pq1.pq1_norm_rope(x, torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        pq1.pq1_norm_rope_grad(x, x, torch.ones(64))
    with pytest.raises(ValueError, match="GPU"):
        pq1.HeadNorm(torch.ones(64))
    with pytest.raises(ValueError, match="weight"):
        pq1.HeadNorm(None)
    u8 = torch.zeros(2, 1, 4, 32, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        pq1.KV4Cache(u8, u8, u8, u8)
    with pytest.raises(TypeError, match="dtype"):
        pq1.KV4Cache(u8, u8, u8, u8, dtype=torch.float32)
    with pytest.raises(ValueError, match="multiple of 32"):
        pq1.KV4Cache.empty(1, 1, 1, 48)
    for call in (pq1.pq1_kv4_append, pq1.pq1_kv_append):
        with pytest.raises(TypeError, match="cache must be"):
            call(None, x, x, None)
    with pytest.raises(TypeError, match="cache must be"):
        pq1.pq1_kv4_read(None, None)


@pytest.mark.parametrize("eps", [0.0, -1.0, math.inf, math.nan, 1e39, 1e-60])
def test_binding_refuses_eps_that_fp32_does_not_hold(eps):
    with pytest.raises(pq1.Pq1Error):
        pq1._need_eps(eps, "test")


@pytest.mark.parametrize("cls,name", [(pq1.KV4Cache, n) for n in ("k", "k_scale", "v", "v_scale")]
                         + [(pq1.HeadNorm, n) for n in ("k_weight", "q_weight")])
def test_tensors_whose_address_is_kept_cannot_be_exchanged(cls, name):
    with pytest.raises(AttributeError):
        setattr(object.__new__(cls), name, torch.zeros(4))


def test_eps_of_a_norm_cannot_be_changed():
    """It went into the struct that the calls pass on."""
    with pytest.raises(AttributeError):
        object.__new__(pq1.HeadNorm).eps = 1e-3


# ---------------------------------------------------------------------------
# The 64-bit forms that the GPU tests rest on
# ---------------------------------------------------------------------------
def test_reference_quantiser_by_hand():
    x = torch.zeros(1, 64)
    x[0, :8] = torch.tensor([7.0, 0.25, 0.75, 1.25, -1.75, 2.5, 3.5, -5.0])
    x[0, 32:36] = torch.tensor([7.5, 0.5, -1.5, 0.49])
    y, byte = ref4.quantise(x, torch.bfloat16)
    assert byte.tolist() == [[127, 128]]
    assert y[0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, -2.0, 2.0, 4.0, -4.0]
    assert y[0, 32:36].tolist() == [8.0, 0.0, -2.0, 0.0]
    x[0, 40] = math.inf
    y, byte = ref4.quantise(x, torch.float16)
    assert byte.tolist() == [[127, 255]] and torch.isnan(y[0, 32:]).all()
    assert ref4.quantise(torch.zeros(1, 32), torch.float16)[1].tolist() == [[104]]
    codes = torch.tensor([[0x21, 0xf7]], dtype=torch.uint8).repeat(1, 8)
    v = ref4.values(codes, torch.tensor([[128]], dtype=torch.uint8))
    assert v[0, :4].tolist() == [1.0, 2.0, 12.0, -12.0]


def test_reference_gradient_by_autograd():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 2, 32, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.randn(32, generator=g, dtype=torch.float64, requires_grad=True)
    gy = torch.randn(3, 2, 32, generator=g, dtype=torch.float64)
    (ref4.norm_rope(x, w, 1e-5)[0] * gy).sum().backward()
    dx, bx, dw, bw = ref4.norm_rope_grad(gy, x.detach(), w.detach(), 1e-5)
    assert torch.allclose(dx, x.grad, atol=1e-12) and torch.allclose(dw, w.grad, atol=1e-12)


def test_struct_sizes():
    assert ctypes.sizeof(pq1.Pq1Kv4Cache) == 56 and ctypes.sizeof(pq1.Pq1HeadNorm) == 24


# Any arguments at all: a code that the header names, and no crash.
weights_any = st.builds(pq1.Pq1HeadNorm, ptr, ptr, st.floats(width=32))
cache4_any = st.builds(pq1.Pq1Kv4Cache, ptr, ptr, ptr, ptr, st.integers(-1, 4), small, size, small, small)


@needs_no_gpu
@settings(**SETTINGS)
@given(x=opt(view), y=opt(view), w=ptr, eps=st.floats(width=32), p=ptr, f=ptr, s=opt(spec_any), T=size,
       H=small, D=small)
def test_norm_any_arguments(lib, x, y, w, eps, p, f, s, T, H, D):  # noqa: F811
    assert lib.pq1_norm_rope(x, y, w, eps, p, f, s, T, H, D, None) in CODES


@needs_no_gpu
@settings(**SETTINGS)
@given(g=opt(view), x=opt(view), d=opt(view), w=ptr, dw=ptr, eps=st.floats(width=32), p=ptr, f=ptr,
       s=opt(spec_any), T=size, H=small, D=small, ws=ptr, n=st.sampled_from([0, 1 << 20, 1 << 40]))
def test_norm_grad_any_arguments(lib, g, x, d, w, dw, eps, p, f, s, T, H, D, ws, n):  # noqa: F811
    assert lib.pq1_norm_rope_grad(g, x, d, w, dw, eps, p, f, s, T, H, D, ws, n, None) in CODES
    assert lib.pq1_norm_rope_grad_workspace_bytes(T, D) >= 0


@needs_no_gpu
@settings(**SETTINGS)
@given(k=opt(view), v=opt(view), sl=ptr, q=opt(view), qo=opt(view), Hq=small, p=ptr, f=ptr,
       s=opt(spec_any), n=opt(weights_any), c=opt(cache_any), c4=opt(cache4_any), T=size)
def test_appends_any_arguments(lib, k, v, sl, q, qo, Hq, p, f, s, n, c, c4, T):  # noqa: F811
    assert lib.pq1_kv_append_ex(k, v, sl, q, qo, Hq, p, f, s, n, c, T, None) in CODES
    assert lib.pq1_kv4_append(k, v, sl, q, qo, Hq, p, f, s, n, c4, T, None) in CODES
    assert lib.pq1_kv4_read(c4, sl, k, v, T, None) in CODES


@needs_no_gpu
@settings(**SETTINGS)
@given(q=opt(view), o=opt(view), c=opt(cache_any), c4=opt(cache4_any), t=ptr, mp=size, cu=ptr, kv=ptr,
       B=size, T=size, Hq=small, mq=size, mkv=size, sc=st.floats(width=32), ca=st.integers(-1, 2), w=small,
       si=small, ws=ptr, n=st.sampled_from([0, 1 << 20, 1 << 40]))
def test_attention_any_arguments(lib, q, o, c, c4, t, mp, cu, kv, B, T, Hq, mq, mkv, sc, ca, w,  # noqa: F811
                                 si, ws, n):
    for fn, of in ((lib.pq1_paged_attention_ex, c), (lib.pq1_kv4_attention, c4)):
        assert fn(q, o, of, t, mp, cu, kv, B, T, Hq, mq, mkv, sc, ca, w, si, ws, n, None) in CODES
        H, D = (of.heads, of.dim) if of is not None else (4, 64)
        assert lib.pq1_paged_attention_ex_workspace_bytes(B, T, Hq, H, D, mq, mkv, w, si) >= 0
        assert lib.pq1_kv4_attention_workspace_bytes(B, T, Hq, H, D, mq, mkv, w, si) >= 0


@needs_no_gpu
@settings(**SETTINGS)
@given(B=st.integers(1, 1 << 23), T=st.integers(1, 1 << 30), Hk=st.integers(1, 1024),
       G=st.integers(1, 64), D=st.sampled_from([64, 128, 256]), mq=st.integers(0, 1 << 62),
       mkv=st.integers(0, 1 << 62), w=st.integers(0, (1 << 31) - 1), si=st.integers(0, (1 << 31) - 1))
def test_attention_plans_of_any_size(lib, B, T, Hk, G, D, mq, mkv, w, si):  # noqa: F811
    """Sizes alone: a plan is refused, or the workspace it asked for does."""
    si = si if w else 0
    views = (heads(1 << 52, n=Hk * G, D=D, hs=D), heads(1 << 53, n=Hk * G, D=D, hs=D))
    rest = (P(1 << 54), 9, P(1 << 55), P(1 << 56), B, T, Hk * G, mq, mkv, 0.1, 1, w, si, P(1 << 57))
    four = pq1.Pq1Kv4Cache(1 << 50, 1 << 48, 1 << 51, 1 << 49, BF16, 16, 9, Hk, D)
    need = lib.pq1_kv4_attention_workspace_bytes(B, T, Hk * G, Hk, D, mq, mkv, w, si)
    assert lib.pq1_kv4_attention(*views, four, *rest, need, None) in (SHAPE, DEVICE)
    need = lib.pq1_paged_attention_ex_workspace_bytes(B, T, Hk * G, Hk, D, mq, mkv, w, si)
    two = cache(n=Hk, D=D, k=1 << 50, v=1 << 51)
    assert lib.pq1_paged_attention_ex(*views, two, *rest, need, None) in (SHAPE, DEVICE)
