"""The attention-layer calls on the GPU against their 64-bit forms: rotation
by positions, the append to a paged cache, attention over the cache."""
import random

import pytest
import torch

import attention_reference as ref

pytestmark = pytest.mark.gpu

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def pq(dev):
    from gemm_hadamard_rotated_amd import pq1
    pq1.load_library()
    return pq1


def check(got, y, bound, where):
    got = got.double().cpu()
    nan = torch.isnan(y)
    assert torch.equal(torch.isnan(got), nan), f"{where}: NaN where none is due, or none where due"
    inf = torch.isinf(y)
    assert torch.equal(got[inf], y[inf]), f"{where}: infinities"
    ok = ~(nan | inf)
    over = ((got - y).abs() - bound)[ok]
    assert over.numel() == 0 or float(over.max()) <= 0, \
        f"{where}: {int((over > 0).sum())} values beyond their bound, worst by {float(over.max()):.3e}"


# ---------------------------------------------------------------------------
# Rotation
# ---------------------------------------------------------------------------
ROPE = [
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
    (70000, 1, 64, 32, (16,), "halves", False, BF16, BF16, 0),
    (3, 2, 1024, 1024, (512,), "adjacent", False, F32, BF16, 12),
    (3000, 8, 72, 18, (9,), "halves", False, BF16, BF16, 0),      # tails at any pair of elements
    (600, 3, 24, 18, (9,), "adjacent", False, F32, F16, 0),       # a tail of six
    (5000, 8, 72, 36, (6, 6, 6), "halves", True, F16, F16, 0),
    (5000, 4, 96, 24, (12,), "adjacent", False, BF16, F32, 0),
]


def positions_of(T, axes, first, seed):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, 1000, (axes, T), generator=g) + first
    return p.clamp(-2 ** 31, 2 ** 31 - 1).to(torch.int32)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", ROPE, ids=lambda c: "-".join(str(v) for v in c[:4]))
def test_rope(pq, dev, case, inverse):
    T, H, D, rot, sections, pairing, inter, din, dout, first = case
    g = torch.Generator().manual_seed(T * 31 + D)
    x = torch.randn(T, H, D, generator=g).to(din)
    pos = positions_of(T, len(sections), first, T)
    freqs = pq.rope_frequencies(rot, 1.0e4)
    rope = pq.Rope(rot, sections, freqs=freqs.to(dev), pairing=pairing, interleaved=inter)
    y = pq.pq1_rope(x.to(dev), pos.to(dev), rope, out_dtype=dout, inverse=inverse)
    assert y.dtype == dout
    e, b = ref.rotate(x, pos, freqs, sections, pairing, inter, inverse)
    check(y, e, ref.rounded_bound(e, b, dout), "rope")
    tail = y[..., rot:].cpu()
    assert torch.equal(tail, x[..., rot:].to(dout)), "elements past rot are copied"


def test_rope_strided_in_place_and_gradient(pq, dev):
    T, H, D, rot = 37, 3, 64, 32
    g = torch.Generator().manual_seed(5)
    stacked = torch.randn(T, 5 * D * H, generator=g).to(dev)
    x = stacked[:, D * H:2 * D * H].unflatten(1, (H, D))
    pos = positions_of(T, 1, 100, 3).to(dev)
    freqs = pq.rope_frequencies(rot)
    rope = pq.Rope(rot, freqs=freqs.to(dev))
    x0 = x.cpu().clone()
    before = stacked.clone()
    e, b = ref.rotate(x0, pos.cpu(), freqs, (16,), "halves", False)
    y = pq.pq1_rope(x, pos[0], rope)                    # [T] positions for one axis
    check(y, e, ref.rounded_bound(e, b, F32), "strided")
    heads_first = torch.randn(H, T, D, generator=g).to(dev).transpose(0, 1)
    out = torch.empty(T, H, 2 * D, device=dev)[..., :D]
    got = pq.pq1_rope(heads_first, pos, rope, out=out)
    assert got is out
    e2, b2 = ref.rotate(heads_first.cpu(), pos.cpu(), freqs, (16,), "halves", False)
    check(out, e2, ref.rounded_bound(e2, b2, F32), "heads first")
    pq.pq1_rope(x, pos, rope, out=x)
    check(x, e, ref.rounded_bound(e, b, F32), "in place")
    assert torch.equal(stacked[:, :D * H], before[:, :D * H])
    assert torch.equal(stacked[:, 2 * D * H:], before[:, 2 * D * H:])
    # The gradient of sum(w * rope(x)) is the inverse rotation of w: against
    # the formula, and against central differences of the 64-bit form.
    w = torch.randn(T, H, D, generator=g)
    grad = pq.pq1_rope(w.to(dev), pos, rope, inverse=True).double().cpu()
    eg, bg = ref.rotate(w, pos.cpu(), freqs, (16,), "halves", False, inverse=True)
    check(grad, eg, ref.rounded_bound(eg, bg, F32), "gradient")
    for t, h, d in ((0, 0, 0), (5, 1, 17), (36, 2, 31), (36, 2, 63)):
        step = torch.zeros(T, H, D, dtype=torch.float64)
        step[t, h, d] = 0.5
        up = ref.rotate(x0 + step, pos.cpu(), freqs, (16,), "halves", False)[0]
        down = ref.rotate(x0 - step, pos.cpu(), freqs, (16,), "halves", False)[0]
        diff = float(((up - down) * w.double()).sum())
        assert abs(float(grad[t, h, d]) - diff) <= 1e-5


@pytest.mark.parametrize("D,rot", [(72, 18), (80, 20), (24, 18), (40, 38), (96, 24), (128, 128)])
@pytest.mark.parametrize("T", [3, 5000])
def test_rope_in_place(pq, dev, T, D, rot):
    x = torch.randn(T, 4, D, generator=torch.Generator().manual_seed(D)).to(BF16).to(dev)
    pos = positions_of(T, 1, 0, 8).to(dev)
    rope = pq.Rope(rot, freqs=pq.rope_frequencies(rot, device=dev))
    want = pq.pq1_rope(x, pos, rope)
    assert torch.equal(pq.pq1_rope(x, pos, rope, out=x), want)


# ---------------------------------------------------------------------------
# Append
# ---------------------------------------------------------------------------
APPEND = [
    (4000, 4, 2, 80, 16, 20, (10,), "halves", False, BF16, BF16),
    (900, 2, 3, 72, 4, 18, (9,), "adjacent", False, F32, F16),
    # T, Hk, G, D, page, rot, sections, pairing, interleaved, in, cache type
    (1, 4, 6, 256, 16, 64, (11, 11, 10), "halves", True, F32, BF16),
    (96, 8, 4, 128, 32, 128, (64,), "halves", False, F16, F16),
    (33, 1, 8, 64, 1, 64, (32,), "adjacent", False, BF16, BF16),
    (700, 2, 7, 80, 8, 20, (10,), "halves", False, F32, F16),
    (50, 4, 0, 64, 128, 64, (8, 12, 12), "adjacent", False, BF16, BF16),
    (21, 3, 2, 40, 4, 0, (), "halves", False, F32, BF16),
    (5, 4, 0, 1024, 2, 0, (), "halves", False, F16, F16),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "-".join(str(v) for v in c[:6]))
def test_append(pq, dev, case):
    T, Hk, G, D, page, rot, sections, pairing, inter, din, dt = case
    g = torch.Generator().manual_seed(T + D)
    pages = -(-T // page) + 3
    qkv = torch.randn(T, (G + 2) * Hk * D, generator=g).to(din)
    cut = qkv.to(dev)
    heads = lambda t, a, n: t[:, a * Hk * D:(a + n) * Hk * D].unflatten(1, (n * Hk, D))
    q, k, v = (heads(cut, 0, G) if G else None), heads(cut, G, 1), heads(cut, G + 1, 1)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 3:      # padding, and slots past either end
        slots[1], slots[2], slots[3] = -1, pages * page, -(2 ** 40)
    cache0 = torch.randn(2, pages, Hk, page, D, generator=g).to(dt)
    cache = pq.KVCache(cache0[0].to(dev), cache0[1].to(dev))
    rope = pos = freqs = None
    if rot:
        freqs = pq.rope_frequencies(rot, 1.0e6)
        rope = pq.Rope(rot, sections, freqs=freqs.to(dev), pairing=pairing, interleaved=inter)
        pos = positions_of(T, len(sections), 4000, 1)
    out = pq.pq1_kv_append(cache, k, v, slots.to(dev), positions=None if pos is None
                           else pos.to(dev), rope=rope, q=q)
    assert (out is None) == (G == 0)

    def turned(x):
        if not rot:
            return x.double(), torch.zeros_like(x, dtype=torch.float64)
        return ref.rotate(x, pos, freqs, sections, pairing, inter)

    ek, bk = turned(heads(qkv, G, 1))
    want_k, want_v = cache0[0].double(), cache0[1].clone()
    bound = torch.zeros_like(want_k)
    for t in range(T):
        s = int(slots[t])
        if 0 <= s < pages * page:
            want_k[s // page, :, s % page] = ek[t]
            bound[s // page, :, s % page] = ref.rounded_bound(ek[t], bk[t], dt)
            want_v[s // page, :, s % page] = heads(qkv, G + 1, 1)[t].to(dt)
    check(cache.k, want_k, bound, "keys")
    assert torch.equal(cache.v.cpu(), want_v), "values are rounded once, other rows untouched"
    if G:
        eq, bq = turned(heads(qkv, 0, G))
        check(out, eq, ref.rounded_bound(eq, bq, dt), "queries")


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
# The longest kv_len that a call states decides, with the number of rows, which
# kernel takes it; any statement has to give right results.
STATED = [1, 10 ** 6]


class Batch:
    """B sequences over a shuffled paged cache; everything unread is NaN."""

    def __init__(self, pq, dev, qs, kvs, Hk, G, D, page, dtype, seed=0, spare=3, peaked=1.5):
        g = torch.Generator().manual_seed(seed * 7919 + D + page)
        self.qs, self.kvs, self.Hk, self.G, self.D, self.page, self.dtype = \
            qs, kvs, Hk, G, D, page, dtype
        need = [-(-n // page) for n in kvs]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g)
        self.table = torch.full((len(qs), max(need) + 2), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.k = [torch.randn(n, Hk, D, generator=g).to(dtype) for n in kvs]
        self.v = [torch.randn(n, Hk, D, generator=g).to(dtype) for n in kvs]
        self.q = (peaked * torch.randn(sum(qs), Hk * G, D, generator=g)).to(dtype)
        self.pages, self.pq, self.dev = pages, pq, dev
        cu = [0]
        for n in qs:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.fill()

    def fill(self):
        """The cache of the present k and v."""
        shape = (self.pages, self.Hk, self.page, self.D)
        kc = torch.full(shape, float("nan"), dtype=self.dtype)
        vc = torch.full(shape, float("nan"), dtype=self.dtype)
        for b, n in enumerate(self.kvs):
            for j in range(0, n, self.page):
                m = min(self.page, n - j)
                p = int(self.table[b, j // self.page])
                if p < 0 or p >= self.pages:
                    continue
                kc[p, :, :m] = self.k[b][j:j + m].transpose(0, 1)
                vc[p, :, :m] = self.v[b][j:j + m].transpose(0, 1)
        self.cache = self.pq.KVCache(kc.to(self.dev), vc.to(self.dev))

    def args(self):
        i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).to(self.dev)
        return self.q.to(self.dev), self.cache, i32(self.table), i32(self.cu), i32(self.kvs)

    def run(self, max_q=None, max_kv=None, **kw):
        return self.pq.pq1_paged_attention(
            *self.args(), max_q=max(self.qs) if max_q is None else max_q,
            max_kv=max(self.kvs) if max_kv is None else max_kv, **kw)

    def check(self, got, causal=True, window=0, scale=None, where="attention"):
        scale = self.D ** -0.5 if scale is None else scale
        for b in range(len(self.qs)):
            q0, q1 = self.cu[b], self.cu[b + 1]
            e, w, spread = ref.attention(self.q[q0:q1], self.k[b], self.v[b], scale, causal, window)
            vmax = float(self.v[b].double().nan_to_num(0, 0, 0).abs().max()) if self.kvs[b] else 0.0
            check(got[q0:q1], e, ref.attention_bound(e, w, spread, self.kvs[b], vmax, self.D,
                                                     self.dtype, got.dtype),
                  f"{where}, sequence {b}")


ATTN = [
    # new tokens, keys, Hk, G, D, page, type, out, causal, window
    ([1], [1], 1, 1, 64, 1, BF16, BF16, True, 0),
    ([1], [2], 1, 8, 128, 16, F16, F32, True, 0),
    ([1, 1, 1], [31, 32, 33], 4, 6, 256, 16, BF16, BF16, True, 0),
    ([1, 1], [700, 129], 4, 6, 256, 64, BF16, F32, True, 0),
    ([1], [5000], 2, 7, 128, 32, F16, F16, True, 0),
    ([1, 1], [900, 300], 2, 16, 64, 8, F16, F32, False, 0),
    ([2, 0, 6, 3], [70, 40, 1, 300], 2, 4, 128, 32, F16, F16, True, 50),   # 6 rows, 1 key
    ([5], [0], 2, 2, 64, 16, BF16, F32, True, 0),                          # no key at all
    ([4, 9], [2, 1000], 8, 1, 256, 1, BF16, BF16, True, 0),
    ([10], [400], 1, 5, 128, 256, BF16, F32, True, 33),
    ([70], [70], 2, 3, 64, 16, BF16, BF16, True, 0),
    ([65, 1, 130], [65, 200, 500], 2, 4, 128, 16, BF16, BF16, True, 0),
    ([100], [1000], 1, 6, 256, 64, BF16, F32, True, 0),
    ([90, 33], [90, 333], 4, 6, 256, 8, F16, F16, True, 40),
    ([129], [300], 2, 4, 128, 1, F16, F32, False, 0),
    ([300, 0, 20], [100, 5, 700], 2, 2, 64, 128, BF16, BF16, True, 0),     # rows without keys
    ([260], [260], 1, 3, 128, 32, BF16, BF16, True, 1),                    # each row sees itself
    ([257], [700], 1, 1, 256, 512, BF16, BF16, True, 100),
    ([64], [4100], 2, 8, 64, 64, F16, F16, True, 0),
]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_attention(pq, dev, case):
    qs, kvs, Hk, G, D, page, dt, dout, causal, window = case
    s = Batch(pq, dev, qs, kvs, Hk, G, D, page, dt)
    for stated in [None] + STATED:
        got = s.run(max_kv=stated, causal=causal, window=window, out_dtype=dout)
        assert got.dtype == dout
        s.check(got, causal, window, where=f"stated {stated}")
        again = s.run(max_kv=stated, causal=causal, window=window, out_dtype=dout)
        assert torch.equal(got, again), "the same call gives the same bits"


def test_attention_scale_and_far_scores(pq, dev):
    # scores of a few hundred: the maximum moves far from tile to tile
    for rows in (1, 3, 100):
        s = Batch(pq, dev, [rows], [640], 1, 2, 64, 16, F16, seed=rows, peaked=6.0)
        s.k[0] *= torch.linspace(0.05, 4.0, 640).view(-1, 1, 1).to(F16)
        s.fill()
        for kv in STATED:
            s.check(s.run(max_kv=kv, scale=0.7, out_dtype=F32), scale=0.7,
                    where=f"{rows} rows, rising")
        s.k[0] = s.k[0].flip(0).contiguous()
        s.fill()
        for kv in STATED:
            s.check(s.run(max_kv=kv, scale=0.7), scale=0.7, where=f"{rows} rows, falling")


@pytest.mark.parametrize("rows,D,out", [(1, 256, BF16), (3, 64, F32), (40, 128, BF16),
                                        (100, 256, BF16), (150, 64, F32)])
def test_attention_strides_and_unowned_rows(pq, dev, rows, D, out):
    s = Batch(pq, dev, [rows, 2], [rows + 77, 9], 2, 3, D, 16, BF16)
    q, cache, table, cu, kv = s.args()
    T = q.shape[0]
    wide = torch.zeros(T + 4, 8 * D * 6, dtype=BF16, device=dev)
    qs = wide[:, D:D + 6 * D].unflatten(1, (6, D))
    qs[2:2 + T] = q
    hold = torch.full((6, T + 4, D + 8), 7.0, dtype=out, device=dev)
    o = hold[:, :, :D].transpose(0, 1)                  # heads outside tokens
    for stated in STATED:
        got = pq.pq1_paged_attention(qs, cache, table, cu + 2, kv, max_q=rows, max_kv=stated, out=o)
        assert got is o
        s.check(o[2:2 + T], where="strided")
    assert bool((hold[:, :2] == 7).all()) and bool((hold[:, T + 2:] == 7).all())
    assert bool((hold[:, :, D:] == 7).all())


@pytest.mark.parametrize("rows", [1, 5, 20, 110])
def test_attention_sizes_beyond_the_hints(pq, dev, rows):
    s = Batch(pq, dev, [rows, rows], [1500, rows], 2, 4, 64, 16, BF16)
    s.check(s.run(), where="true hints")
    s.check(s.run(max_q=1, max_kv=1), where="hints too small")
    s.check(s.run(max_q=4 * rows, max_kv=9000), where="hints too large")
    s.check(s.run(max_q=1, max_kv=10 ** 6), where="one hint too small, one too large")
    s.check(s.run(max_q=4 * rows, max_kv=1), where="one hint too large, one too small")


@pytest.mark.parametrize("D", [64, 256])
def test_attention_more_pages_than_a_workgroup_holds(pq, dev, D):
    """Pages of one key: the page numbers of a part are taken in pieces."""
    s = Batch(pq, dev, [20, 17], [9000, 4100], 1, 2, D, 1, BF16)
    for stated in STATED + [2 * 10 ** 6, 10 ** 9]:
        s.check(s.run(max_kv=stated), where=f"stated {stated}")
    s = Batch(pq, dev, [33], [9000], 1, 2, D, 1, BF16, seed=1)
    for stated in (2 * 10 ** 6, 10 ** 9):
        s.check(s.run(max_kv=stated, window=6000), window=6000, where=f"stated {stated}")


@pytest.mark.parametrize("page,dt", [(16, BF16), (64, F16), (4, BF16)])
@pytest.mark.parametrize("rows,D", [(1, 64), (4, 128), (30, 256), (120, 128), (70, 64)])
def test_attention_odd_values(pq, dev, rows, D, page, dt):
    """Infinities and NaN in values reach the rows that see them, and no
    others; in keys likewise."""
    kv = rows + 150
    for what in ("value", "key"):
        s = Batch(pq, dev, [rows], [kv], 1, 2, D, page, dt, seed=3)
        if what == "value":
            s.v[0][kv - 1, 0, 5] = float("nan")              # only the last token sees it
            s.v[0][kv - 1, 0, 6] = float("inf")
            s.v[0][kv - max(1, rows // 2), 0, 9] = float("-inf")
        else:
            s.k[0][kv - 1, 0, 1] = float("nan")
        s.fill()
        for out in (dt, F32):
            for stated in STATED:
                s.check(s.run(max_kv=stated, out_dtype=out), where=f"odd {what}, stated {stated}")
    s = Batch(pq, dev, [rows], [kv], 1, 2, D, page, dt, seed=4)
    s.v[0][20, 0, 3] = float("inf")                           # before every row's window
    s.k[0][21] = float("nan")
    s.fill()
    for stated in STATED:
        s.check(s.run(max_kv=stated, window=90), window=90, where="outside the window")


@pytest.mark.parametrize("stated", STATED)
@pytest.mark.parametrize("page", [8, 32, 128])
@pytest.mark.parametrize("rows", [1, 6, 90])
def test_attention_bad_pages(pq, dev, rows, page, stated):
    """A page outside the cache makes NaN of the rows that see it, and
    nothing else is read; a page that a window has left may be anything."""
    kv = rows + 300
    s = Batch(pq, dev, [rows, 3], [kv, 40], 2, 4, 64, page, BF16)
    want = s.run(max_kv=stated)
    last = (kv - 1) // page
    good = int(s.table[0, last])
    for bad in (-1, s.pages, 2 ** 31 - 1, -2 ** 31):
        s.table[0, last] = bad
        got = s.run(max_kv=stated)
        sees = torch.arange(rows) + kv - rows >= last * page
        assert bool(torch.isnan(got[:rows].cpu()[sees]).all())
        assert not bool(torch.isnan(got[:rows].cpu()[~sees]).any())
        assert torch.equal(got[rows:], want[rows:])
        s.table[0, last] = good
    short = s.pq.pq1_paged_attention(*(a if i != 2 else a[:, :last].contiguous()
                                       for i, a in enumerate(s.args())), max_q=rows, max_kv=stated)
    assert torch.equal(torch.isnan(short[:rows]).all(-1).all(-1).cpu(),
                       torch.arange(rows) + kv - rows >= last * page)
    want = s.run(max_kv=stated, window=100)
    left = (kv - rows + 1 - 100) // page                     # pages no window reaches
    if left > 0:
        s.table[0, :left] = -1
        assert torch.equal(s.run(max_kv=stated, window=100), want)


def test_attention_lengths_outside_their_range(pq, dev):
    s = Batch(pq, dev, [2, 3, 1], [50, 20, 9], 2, 2, 64, 16, BF16)
    q, cache, table, cu, kv = s.args()
    want = s.run()
    got = torch.full_like(want, 5)
    bad_cu = torch.tensor([-7, 2, 1, 900], dtype=torch.int32, device=dev)   # 0-2, none, 1-6
    pq.pq1_paged_attention(q, cache, table, bad_cu, torch.tensor([50, -3, 0], dtype=torch.int32,
                                                                 device=dev),
                           max_q=6, max_kv=50, out=got)
    assert torch.equal(got[:1], want[:1])
    assert bool((got[2:] == 0).all())


def test_attention_far_into_a_large_cache(pq, dev):
    """Element offsets past 2^31 and byte offsets past 2^32."""
    Hk, page, D = 8, 64, 128
    pages = (1 << 32) // (Hk * page * D) + 40
    kc = torch.empty((pages, Hk, page, D), dtype=BF16, device=dev)
    vc = torch.empty((pages, Hk, page, D), dtype=BF16, device=dev)
    for rows, stated in ((1, 200), (40, 200), (40, 10 ** 6)):
        s = Batch(pq, dev, [rows], [200], Hk, 2, D, page, BF16)
        far = torch.tensor([pages - 1, 3, pages - 7, pages // 2 + 1])
        for i, p in enumerate(far.tolist()):
            kc[p], vc[p] = s.cache.k[int(s.table[0, i])], s.cache.v[int(s.table[0, i])]
        s.table[0, :4] = far.to(torch.int32)
        s.cache = pq.KVCache(kc, vc)
        s.check(s.run(max_kv=stated), where="large cache")
    new = torch.randn(2, Hk, D, dtype=BF16, device=dev)
    slots = torch.tensor([pages * page - 1, (pages - 2) * page + 5], device=dev)
    pq.pq1_kv_append(s.cache, new, new, slots)
    assert torch.equal(kc[pages - 1, :, page - 1], new[0])
    assert torch.equal(vc[pages - 2, :, 5], new[1])


def test_attention_layer_on_a_side_stream_and_in_a_graph(pq, dev):
    """Append and attention of one decoded token captured into a graph: each
    replay reads the present inputs, with eager work in between."""
    s = Batch(pq, dev, [1, 1, 1], [600, 65, 1300], 4, 6, 256, 16, BF16)
    q, cache, table, cu, kv = s.args()
    freqs = pq.rope_frequencies(64, 1.0e6).to(dev)
    rope = pq.Rope(64, (11, 11, 10), freqs=freqs, interleaved=True)
    qkv = torch.randn(3, 32 * 256, device=dev)
    qx, kx, vx = (qkv[:, a * 256:b * 256].unflatten(1, (b - a, 256))
                  for a, b in ((0, 24), (24, 28), (28, 32)))
    pos = torch.zeros(3, 3, dtype=torch.int32, device=dev)
    slots = torch.zeros(3, dtype=torch.int64, device=dev)

    def step():
        qr = pq.pq1_kv_append(cache, kx, vx, slots, positions=pos, rope=rope, q=qx)
        return pq.pq1_paged_attention(qr, cache, table, cu, kv, max_q=1, max_kv=2000)

    def inputs(i):
        g = torch.Generator(device=dev).manual_seed(i)
        qkv.copy_(torch.randn(3, 32 * 256, device=dev, generator=g))
        lens = torch.tensor([600 - i, 65 - i, 1300 - i], device=dev)
        kv.copy_(lens)
        pos.copy_((lens - 1).expand(3, 3))
        at = lens - 1
        slots.copy_(table[torch.arange(3, device=dev), at // 16].long() * 16 + at % 16)

    side = torch.cuda.Stream()
    inputs(0)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step()
    side.synchronize()
    assert torch.equal(first, step())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(1, 6):
        inputs(i)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step()), f"replay {i}"


def test_example_layer(pq, dev):
    """Chunks and single tokens give what the whole prompt gives.  Both round
    activations, probabilities and queries to bf16 (2^-8 each; single tokens do
    not round the projection's input), so outputs differ by a few times 2^-8 of
    their size."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import attention_layer as ex
    layer = ex.AttentionLayer(hidden=1024, heads=4, kv_heads=2, dim=256, pages=40, page_size=16)
    x = torch.randn(150, 1024, device=dev, generator=torch.Generator(device=dev).manual_seed(1))
    whole = ex.run(layer, x, range(10), [150])
    parts = ex.run(layer, x, range(30, 20, -1), [64, 1, 50, 33, 1, 1])
    size = whole.double().pow(2).mean().sqrt()
    assert float((parts - whole).double().pow(2).mean().sqrt()) <= 8 * 2 ** -8 * float(size)
    # the layer against its 64-bit form, from the projection's output on
    D, seq = 256, ex.Sequence(layer, range(10))
    a = seq.extend(150)
    qkv = layer._project(x, layer.qkv)
    q, k, v = (qkv[:, i * D:j * D].unflatten(1, (j - i, D)) for i, j in ((0, 4), (4, 6), (6, 8)))
    qr = pq.pq1_kv_append(layer.cache, k, v, a["slots"], positions=a["positions"], rope=layer.rope,
                          q=q)
    o = pq.pq1_paged_attention(qr, layer.cache, a["table"], a["cu_q"], a["kv_len"], 150, 150,
                               out_dtype=F32)
    f = layer.rope.freqs.cpu()
    kr, _ = ref.rotate(k.cpu(), a["positions"].cpu(), f, (11, 11, 10), "halves", True)
    e, w, spread = ref.attention(qr.cpu(), kr.to(BF16), v.cpu().to(BF16), D ** -0.5, True, 0)
    # a key may round to the other neighbour: two bf16 steps of every score
    b = ref.attention_bound(e, w, spread, 150, 0.0, D, BF16, F32) + 2 * w * 2 ** -7 * spread
    check(o, e, b, "example")


def test_binding_refusals(pq, dev):
    """Raised before anything is launched."""
    s = Batch(pq, dev, [2], [40], 2, 2, 64, 16, BF16)
    q, cache, table, cu, kv = s.args()
    att = lambda *a, **k: pq.pq1_paged_attention(*a, max_q=2, max_kv=40, **k)
    with pytest.raises(TypeError):
        att(q.float(), cache, table, cu, kv)
    with pytest.raises(ValueError):
        att(q[..., :32].contiguous(), cache, table, cu, kv)
    with pytest.raises(ValueError):
        att(q.transpose(1, 2).contiguous().transpose(1, 2), cache, table, cu, kv)
    with pytest.raises(TypeError):
        att(q, cache, table.long(), cu, kv)
    with pytest.raises(ValueError):
        att(q, cache, table, cu[:1], kv)
    with pytest.raises(ValueError):
        att(q, cache, table[:, ::2], cu, kv)
    with pytest.raises(ValueError):
        att(q, cache, table.cpu(), cu, kv)
    with pytest.raises(TypeError):
        att(q, cache, table, cu, kv, out_dtype=F16)
    with pytest.raises(ValueError):
        att(q, cache, table, cu, kv, out=torch.empty(3, 4, 64, dtype=BF16, device=dev))
    with pytest.raises(pq.Pq1Error):
        att(q[:, :3].contiguous(), cache, table, cu, kv)          # 3 heads over 2
    with pytest.raises(pq.Pq1Error):
        att(q, cache, table, cu, kv, scale=-1.0)
    with pytest.raises(pq.Pq1Error):
        att(q, cache, table, cu, kv, causal=False, window=3)
    with pytest.raises(pq.Pq1Error):
        att(q, cache, table, cu, kv, out=q)
    odd = pq.KVCache(torch.zeros(2, 1, 24, 64, dtype=BF16, device=dev),
                     torch.zeros(2, 1, 24, 64, dtype=BF16, device=dev))
    with pytest.raises(pq.Pq1Error):
        att(q, odd, table, cu, kv)                                # pages of 24
    rope = pq.Rope(32, (8, 8), freqs=pq.rope_frequencies(32, device=dev))
    pos = torch.zeros(2, 2, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        pq.pq1_rope(q, pos[:1], rope)
    with pytest.raises(TypeError):
        pq.pq1_rope(q, pos.long(), rope)
    with pytest.raises(pq.Pq1Error):
        pq.pq1_rope(q[..., :24].contiguous(), pos, rope)          # 32 elements of 24
    for bad in (dict(rot=31), dict(rot=32, sections=(8, 9)), dict(rot=32, sections=(4,) * 5),
                dict(rot=32, pairing="thirds")):
        with pytest.raises(pq.Pq1Error):
            pq.Rope(freqs=pq.rope_frequencies(bad["rot"], device=dev), **bad)
    new, slots = torch.zeros(2, 2, 64, dtype=BF16, device=dev), torch.arange(2, device=dev)
    with pytest.raises(ValueError):
        pq.pq1_kv_append(cache, new, new, slots[:1])
    with pytest.raises(TypeError):
        pq.pq1_kv_append(cache, new, new.float(), slots)
    with pytest.raises(ValueError):
        pq.pq1_kv_append(cache, new, new, slots, rope=rope)
    with pytest.raises(ValueError):
        pq.pq1_kv_append(cache, new, new, slots, q_out=new)
    with pytest.raises(ValueError):
        pq.pq1_kv_append(cache, new[:, :1], new[:, :1], slots)


def test_empty_calls(pq, dev):
    s = Batch(pq, dev, [0, 0], [5, 0], 2, 2, 64, 16, BF16)
    assert s.run().shape == (0, 4, 64)
    rope = pq.Rope(32, freqs=pq.rope_frequencies(32, device=dev))
    none = torch.empty(0, 2, 64, dtype=BF16, device=dev)
    pos = torch.empty(0, dtype=torch.int32, device=dev)
    assert pq.pq1_rope(none, pos, rope).shape == (0, 2, 64)
    got = pq.pq1_kv_append(s.cache, none, none, pos.long(), positions=pos, rope=rope, q=none)
    assert got.shape == (0, 2, 64)
