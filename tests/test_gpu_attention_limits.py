"""The attention-layer calls on the GPU at the edges of what they allow: hints
of any size, chunks and caches beyond the hints, values and probabilities at the
ends of their types' ranges, workspaces in graphs."""
import pytest
import torch

import attention_reference as ref
from test_gpu_attention import BF16, F16, F32, Batch, check, pq  # noqa: F401  (pq: fixture)

pytestmark = pytest.mark.gpu


def attention_rows(q, k, v, scale, causal=True):
    """ref.attention for finite inputs of which every row sees a key: all rows
    of a head at once."""
    q, k, v = q.double(), k.double(), v.double()
    n, kv, G = q.shape[0], k.shape[0], q.shape[1] // k.shape[1]
    o, weight, spread = torch.zeros_like(q), torch.zeros_like(q), 0.0
    for h in range(q.shape[1]):
        K, V = k[:, h // G], v[:, h // G]
        e = (q[:, h] @ K.t()) * scale
        spread = max(spread, float((q[:, h].abs() @ K.abs().t()).max()) * scale)
        if causal:
            e.masked_fill_(~torch.ones(n, kv, dtype=torch.bool).tril(kv - n), -float("inf"))
        p = torch.softmax(e, dim=1)
        o[:, h], weight[:, h] = p @ V, p @ V.abs()
    return o, weight, spread


def check_rows(s, got, where, causal=True):
    """Batch.check of one sequence by attention_rows."""
    e, w, spread = attention_rows(s.q, s.k[0], s.v[0], s.D ** -0.5, causal)
    check(got, e, ref.attention_bound(e, w, spread, s.kvs[0], float(s.v[0].abs().max()), s.D,
                                      s.dtype, got.dtype), where)


@pytest.mark.parametrize("stated", [0x7fff0000, 0x7fffff01, 2 ** 31 - 1, 2 ** 62])
@pytest.mark.parametrize("B,rows,G", [(64, 1, 6), (1, 150, 8), (2, 1, 2)])
def test_longest_cache_stated_without_limit(pq, dev, B, rows, G, stated):
    """A caller that knows no limit states the largest number."""
    Hk = 4 if B > 1 else 32
    kvs = [rows + 9 + 3 * (b % 5) for b in range(B)]
    s = Batch(pq, dev, [rows] * B, kvs, Hk, G, 64, 16, BF16)
    if B == 1:
        check_rows(s, s.run(max_kv=stated), f"stated {stated}")
    else:
        s.check(s.run(max_kv=stated), where=f"stated {stated}")


@pytest.mark.parametrize("kv", [2300, 2810, 3320])
@pytest.mark.parametrize("D,G,dt", [(64, 4, BF16), (128, 4, F16), (128, 2, BF16), (256, 2, BF16)])
def test_many_rows_in_parts_longer_than_stated(pq, dev, D, G, dt, kv):
    """A prompt chunk whose keys are cut (8 parts of 256 keys are planned), on a
    cache that has grown past the stated 2048 keys."""
    s = Batch(pq, dev, [1024 // G], [kv], 8, G, D, 16, dt)
    assert pq.load_library().pq1_paged_attention_workspace_bytes(
        1, 1024 // G, 8 * G, 8, D, 1024 // G, 2048) == 8 * 1024 * 8 * (4 * D + 8)
    check_rows(s, s.run(max_kv=2048), f"{kv} keys")
    check_rows(s, s.run(max_kv=2048, causal=False), f"{kv} keys, all seen", causal=False)


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows,kv,max_kv", [(40, 120, 1), (90, 90, 1), (70, 4000, 10 ** 6),
                                            (33, 20, 1), (200, 3, 400)])
def test_odd_values_in_chunks_longer_than_stated(pq, dev, rows, kv, max_kv, out):
    """A workgroup that walks over several row tiles, infinities and NaN among
    the values of some of them (and rows without a key)."""
    s = Batch(pq, dev, [rows, 3], [kv, 50], 2, 4, 64, 16, BF16, seed=rows)
    s.v[0][kv - 1, 0, 5] = float("nan")
    s.v[0][kv - 1, 1, 6] = float("inf")
    s.v[0][kv // 2, 0, 9] = float("-inf")
    s.v[1][48, 1, 2] = float("inf")
    s.fill()
    for max_q in (1, 5):
        s.check(s.run(max_q=max_q, max_kv=max_kv, out_dtype=out), where=f"stated {max_q} rows")


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("B,rows,stated", [(1, 1, 1), (1, 20, 1), (130, 256, 8192)])
def test_many_small_probabilities_of_f16(pq, dev, B, rows, stated, D):
    """A first key of probability 1 and value 0, then n = 2^11 keys of 2^-20 and
    value 1, all met by the same wave in one part (tiles of 32 keys, every
    fourth; the keys between are far below); fp32 result n 2^-20 / (1 + n 2^-20).

    An f16 probability is taken to the nearest 2^-32 of the largest, so each is
    off by at most 2^-33: n 2^-33 in all.  The 32-bit sum of the probabilities
    begins at the largest; a lane adds at most n / 2 times to it, each time off
    by 2^-24 of it: n 2^-25 of the result, which is n 2^-20.  The numerator stays
    below n 2^-20 (n / 16 additions, 2^-25 of that each), the exponential is good
    to 2^-21, its argument to 2^-20, the result is rounded once."""
    page, n = 256, 2 ** 11
    kv = 4 * n
    ln2 = torch.tensor(2.0, dtype=torch.float64).log()
    hi = (-20 * ln2).to(F16)
    lo = ((-20 * ln2 - hi.double()) * 2 ** 8).to(F16)
    w = float(torch.exp(hi.double() + lo.double() * 2.0 ** -8))
    assert abs(w * 2 ** 20 - 1) < 2.0 ** -18
    small = torch.arange(kv, device=dev) // 32 % 4 == 0
    small[0] = False
    k = torch.zeros(kv, D, dtype=F16, device=dev)
    k[:, 0] = torch.where(small, hi.to(dev), torch.tensor(-60000.0, dtype=F16, device=dev))
    k[:, 1] = torch.where(small, lo.to(dev), torch.zeros((), dtype=F16, device=dev))
    k[0] = 0
    v = small.to(F16).unsqueeze(1).expand(kv, D)
    paged = lambda x: x.reshape(kv // page, 1, page, D).contiguous()
    q = torch.zeros(B * rows, 1, D, dtype=F16, device=dev)
    q[..., 0], q[..., 1] = 1.0, 2.0 ** -8
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    table = torch.arange(kv // page, dtype=torch.int32, device=dev).expand(B, -1).contiguous()
    got = pq.pq1_paged_attention(q, pq.KVCache(paged(k), paged(v)), table,
                                 i32([b * rows for b in range(B + 1)]), i32([kv] * B), max_q=rows,
                                 max_kv=stated, scale=1.0, causal=False, out_dtype=F32).double()
    share = (n - 1) * w
    o = share / (1 + share)
    bound = n * 2.0 ** -33 + o * (n * 2.0 ** -25 + n / 16 * 2.0 ** -25 + 2.0 ** -20 + 2.0 ** -21
                                  + 2.0 ** -24)
    worst = float((got - o).abs().max())
    assert worst <= bound, f"off by {worst:.3e}, bound {bound:.3e}"


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows,kv,D", [(1, 1, 64), (1, 3000, 256), (5, 700, 128), (90, 900, 64),
                                       (300, 300, 256)])
def test_largest_finite_values(pq, dev, rows, kv, D, out):
    """bf16 values up to the largest number: their average is finite."""
    s = Batch(pq, dev, [rows], [kv], 1, 2, D, 16, BF16, seed=kv)
    s.v[0] = (s.v[0].sign() * 1.5 * 2.0 ** 120).to(BF16)
    s.v[0][..., ::3] = torch.finfo(BF16).max
    s.v[0][..., 1::3] = -torch.finfo(BF16).max
    s.fill()
    for stated in (1, kv, 10 ** 6):
        check_rows(s, s.run(max_kv=stated, out_dtype=out), f"stated {stated}")


@pytest.mark.parametrize("out", [BF16, F32])
@pytest.mark.parametrize("rows", [1, 90])
def test_small_values(pq, dev, rows, out):
    """Values near the small end of bf16: products keep the bits of fp32 down to
    2^-149, which is 2^-129 of a probability of one (one such loss a product)."""
    s = Batch(pq, dev, [rows], [400], 1, 2, 64, 16, BF16, seed=2)
    s.v[0] = (s.v[0].double() * 2.0 ** -110).to(BF16)
    s.fill()
    for stated in (1, 10 ** 6):
        got = s.run(max_kv=stated, out_dtype=out)
        e, w, spread = attention_rows(s.q, s.k[0], s.v[0], s.D ** -0.5)
        b = ref.attention_bound(e, w, spread, 400, 0.0, 64, BF16, out) + 3 * 400 * 2.0 ** -129
        check(got, e, b, f"stated {stated}")


def test_numbers_past_their_c_types(pq, dev):
    """A window, or a number of heads, is not taken by its low 32 bits."""
    s = Batch(pq, dev, [3], [90], 2, 2, 64, 16, BF16)
    want = s.run()
    for window in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5):
        assert torch.equal(s.run(window=window), want), window
    with pytest.raises(pq.Pq1Error):
        s.run(window=5 - 2 ** 32)
    assert torch.equal(s.run(max_q=2 ** 64 + 1, max_kv=2 ** 63), s.run(max_q=2 ** 62, max_kv=2 ** 62))
    rope = pq.Rope(8, freqs=pq.rope_frequencies(8, device=dev))
    pos = torch.zeros(1, dtype=torch.int32, device=dev)
    one = torch.zeros(1, 1, 8, dtype=BF16, device=dev)
    with pytest.raises(ValueError, match="32-bit"):
        pq.pq1_rope(one.expand(1, 2 ** 32 + 1, 8), pos, rope)
    with pytest.raises(ValueError, match="32-bit"):
        pq.pq1_kv_append(s.cache, s.cache.k[0, :, :1].transpose(0, 1), s.cache.v[0, :, :1].transpose(
            0, 1), pos.long(), q=one.repeat(1, 1, 8).expand(1, 2 ** 32 + 1, 64))


def test_graphs_of_one_capture_stream_replayed_on_two(pq, dev):
    """Each graph has its own partial sums: replayed at the same time on two
    streams, with calls of its own on a third, every result is the eager one."""
    batches = [Batch(pq, dev, [1], [60000 + 100 * i], 4, 6, 256, 64, BF16, seed=i) for i in range(3)]
    args = [b.args() for b in batches]
    call = lambda i, **k: pq.pq1_paged_attention(*args[i], max_q=1, max_kv=60000 + 100 * i, **k)
    want = [call(i).clone() for i in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i))
        graphs.append(g)
    for turn in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(20):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
            third = call(2)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i]), f"graph {i}, turn {turn}"
        assert torch.equal(third, want[2])


def test_rotation_past_one_launch(pq, dev):
    """2^34 elements in pieces of two are more workgroups than a launch holds."""
    H, D, T = 1024, 8, 2 ** 21 + 5
    x = torch.randn(1, H, D, generator=torch.Generator().manual_seed(1)).to(BF16).to(dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    rope = pq.Rope(2, freqs=torch.tensor([0.37], dtype=torch.float64, device=dev))
    y = torch.full((T, H, D), 7.0, dtype=BF16, device=dev)
    pq.pq1_rope(x.expand(T, H, D), pos, rope, out=y)
    some = torch.tensor([0, 1, 2 ** 20, 2 ** 21 - 2, 2 ** 21 - 1, 2 ** 21, T - 2, T - 1], device=dev)
    want = pq.pq1_rope(x.expand(8, H, D), pos[some].contiguous(), rope)
    assert torch.equal(y[some], want)
    assert not bool((y[:, :, 2:] == 7.0).all(-1).all(-1).any())      # no token left out
    del y
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dt,size,scale", [(F16, 2.0 ** 14.3, 0.7), (F16, 2.0 ** 14.3, 50.0),
                                           (BF16, 2.0 ** 21.7, 0.1), (BF16, 2.0 ** 40.2, 3.0)])
@pytest.mark.parametrize("rows,D", [(1, 256), (5, 64), (90, 128), (40, 256), (300, 64)])
def test_scores_past_the_steps_of_fp32(pq, dev, dt, size, scale, rows, D):
    """Scores of which neighbouring floats are further apart than 1: the largest
    takes all, equal ones share, whatever the sign.  (Scores here differ by 2^-6
    of themselves, far more than their rounding, 2^-24 of themselves.)"""
    kv = 700
    s = Batch(pq, dev, [rows], [kv], 1, 2, D, 16, dt, seed=D)
    g = torch.Generator().manual_seed(rows)
    for sign in (1.0, -1.0):
        s.q = torch.zeros(rows, 2, D, dtype=dt)
        s.q[:, 0, 0], s.q[:, 1, 0] = size, size / 2
        level = torch.randint(1, 60, (kv,), generator=g)       # larger level, larger score
        s.k[0] = torch.zeros(kv, 1, D, dtype=dt)
        step = level if sign > 0 else 61 - level
        s.k[0][:, 0, 0] = sign * size * (0.03 * step.double()).to(dt)
        s.fill()
        k0 = sign * s.k[0][:, 0, 0].double()
        order = k0 if sign > 0 else -k0
        o = torch.zeros(rows, 2, D, dtype=torch.float64)
        for i in range(rows):
            sees = order[:kv - rows + i + 1]
            top = sees == sees.max()
            o[i] = s.v[0][:kv - rows + i + 1, 0][top].double().mean(0)
        for out in (dt, F32):
            for stated in (1, kv, 10 ** 6):
                got = s.run(max_kv=stated, scale=scale, out_dtype=out)
                # equal probabilities: sums in 32 bits, a rounding to the type
                b = o.abs() * 0 + kv * 2.0 ** -23 * 5
                check(got, o, ref.rounded_bound(o, b, out), f"sign {sign}, stated {stated}")
