"""Attention over a 4-bit cache, and in windows whose first keys stay visible (over
caches of either kind), on the GPU against 64-bit forms."""
import random

import pytest
import torch

import attention_reference as ref
import kv4_reference as ref4
from test_gpu_attention import ATTN, BF16, F16, F32, STATED, Batch, check, pq  # noqa: F401

pytestmark = pytest.mark.gpu


class Pages(Batch):
    """A batch over a 16-bit cache, in windows with first keys."""

    def run(self, max_q=None, max_kv=None, **kw):
        return self.call(*self.args(), max_q=max(self.qs) if max_q is None else max_q,
                         max_kv=max(self.kvs) if max_kv is None else max_kv, **kw)

    @property
    def call(self):
        return self.pq.pq1_paged_attention

    def check(self, got, causal=True, window=0, sinks=0, scale=None, where="attention", rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        for b in range(len(self.qs)):
            q0, q1 = self.cu[b], self.cu[b + 1]
            if rows is not None:            # of each sequence, counted from its end
                q0 = max(q0, q1 - rows)
            e, w, spread = ref4.attention(self.q[q0:q1], self.k[b], self.v[b], scale, causal, window,
                                          sinks)
            vmax = float(self.v[b].double().nan_to_num(0, 0, 0).abs().max()) if self.kvs[b] else 0.0
            check(got[q0:q1], e, ref.attention_bound(e, w, spread, self.kvs[b], vmax, self.D,
                                                     self.dtype, got.dtype),
                  f"{where}, sequence {b}")


class Pages4(Pages):
    """The same over a 4-bit cache; k and v become what it holds, and every byte that
    holds none of them is 255 (NaN, as a scale)."""

    @property
    def call(self):
        return self.pq.pq1_kv4_attention

    def fill(self):
        shape = (self.pages, self.Hk, self.page)
        made = []
        for x in (self.k, self.v):
            codes = torch.full((*shape, self.D // 2), 255, dtype=torch.uint8)
            scales = torch.full((*shape, self.D // 32), 255, dtype=torch.uint8)
            for b, n in enumerate(self.kvs):
                y, byte = ref4.quantise(x[b], self.dtype)
                x[b] = y.to(self.dtype)
                assert torch.equal(x[b].double().nan_to_num(9), y.nan_to_num(9))
                c = ref4.encode(y.nan_to_num(0), byte)
                for j in range(0, n, self.page):
                    m = min(self.page, n - j)
                    p = int(self.table[b, j // self.page])
                    codes[p, :, :m] = c[j:j + m].transpose(0, 1)
                    scales[p, :, :m] = byte[j:j + m].transpose(0, 1)
            made += [codes.to(self.dev), scales.to(self.dev)]
        self.cache = self.pq.KV4Cache(*made, dtype=self.dtype)


KINDS = [Pages, Pages4]
IDS = ["16 bits", "4 bits"]


@pytest.mark.parametrize("case", ATTN, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_attention4(pq, dev, case):  # noqa: F811
    qs, kvs, Hk, G, D, page, dt, dout, causal, window = case
    s = Pages4(pq, dev, qs, kvs, Hk, G, D, page, dt)
    for stated in [None] + STATED:
        got = s.run(max_kv=stated, causal=causal, window=window, out_dtype=dout)
        assert got.dtype == dout
        s.check(got, causal, window, where=f"stated {stated}")
        again = s.run(max_kv=stated, causal=causal, window=window, out_dtype=dout)
        assert torch.equal(got, again), "the same call gives the same bits"


WINDOWS = [
    # new tokens, keys, Hk, G, D, page, type, out, window, sinks
    ([1], [1], 1, 1, 64, 1, BF16, BF16, 1, 1),
    ([1, 1, 1], [500, 64, 3], 4, 6, 256, 16, BF16, BF16, 100, 4),
    ([1, 1], [1500, 700], 8, 4, 128, 32, F16, F16, 257, 65),
    ([1], [900], 1, 8, 64, 1, F16, F32, 7, 130),
    ([1], [3000], 2, 7, 128, 4, BF16, F32, 1, 1),
    ([4, 0, 6, 3], [70, 40, 1, 700], 2, 4, 128, 32, F16, F16, 50, 5),       # 6 rows, 1 key
    ([7], [300], 2, 2, 256, 64, BF16, F32, 32, 64),
    ([5], [400], 1, 5, 128, 256, BF16, BF16, 33, 399),                      # nearly all of them
    ([5], [400], 1, 5, 128, 16, BF16, BF16, 33, 1000),                      # more than there are
    ([90], [300], 2, 3, 64, 16, BF16, BF16, 64, 1),
    ([130, 2], [500, 260], 2, 4, 128, 16, BF16, BF16, 70, 20),
    ([100], [1000], 1, 6, 256, 64, BF16, F32, 128, 128),
    ([70], [900], 1, 6, 64, 64, F16, F16, 1, 3),
    ([129], [420], 2, 4, 128, 1, F16, F32, 60, 90),
    ([300], [280], 1, 2, 64, 128, BF16, BF16, 90, 17),                      # rows without keys
    ([257], [700], 1, 1, 256, 512, BF16, BF16, 100, 33),
]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: "-".join(str(v) for v in c).replace(" ", ""))
def test_first_keys_in_windows(pq, dev, case, kind):  # noqa: F811
    qs, kvs, Hk, G, D, page, dt, dout, window, sinks = case
    s = kind(pq, dev, qs, kvs, Hk, G, D, page, dt)
    # from the present length both ways: hints decide the kernel and the parts
    for stated in [None] + STATED:
        got = s.run(max_kv=stated, window=window, sinks=sinks, out_dtype=dout)
        s.check(got, True, window, sinks, where=f"stated {stated}")
        again = s.run(max_kv=stated, window=window, sinks=sinks, out_dtype=dout)
        assert torch.equal(got, again), "the same call gives the same bits"
    s.check(s.run(max_q=1, max_kv=10 ** 6, window=window, sinks=sinks), True, window, sinks,
            where="one hint too small")
    s.check(s.run(max_q=5 * max(qs), max_kv=1, window=window, sinks=sinks), True, window, sinks,
            where="one hint too large")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_first_keys_drawn(pq, dev, kind):  # noqa: F811
    """Sizes at random, first keys and windows around the sizes of tiles and pages."""
    rng = random.Random(7)
    for turn in range(60):
        D, page = rng.choice([64, 128, 256]), rng.choice([1, 2, 8, 16, 32, 64, 128])
        B = rng.choice([1, 1, 2, 3])
        n = rng.choice([1, 1, 2, 5, 17, 40])
        qs = [rng.randint(1, n) for _ in range(B)]
        kvs = [q + rng.choice([0, 3, rng.randint(0, 400)]) for q in qs]
        window = rng.choice([1, 31, 32, 64, 65, rng.randint(1, 300)])
        sinks = rng.choice([1, 4, 32, 63, 64, 65, rng.randint(1, 300)])
        s = kind(pq, dev, qs, kvs, rng.choice([1, 2]), rng.choice([1, 3, 8]), D, page,
                 rng.choice([BF16, F16]), seed=turn)
        stated = rng.choice([None, 1, 10 ** 6])
        got = s.run(max_kv=stated, window=window, sinks=sinks, out_dtype=rng.choice([None, F32]))
        s.check(got, True, window, sinks, where=f"turn {turn}, {qs} {kvs} {D} {page} {window} {sinks}")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("rows", [1, 5, 40, 110])
def test_pages_between_first_keys_and_window_are_not_read(pq, dev, rows, kind):  # noqa: F811
    kv, page, window, sinks = rows + 700, 16, 60, 20
    s = kind(pq, dev, [rows, 2], [kv, 40], 2, 4, 64, page, BF16)
    for stated in STATED:
        want = s.run(max_kv=stated, window=window, sinks=sinks)
        assert not bool(torch.isnan(want).any())
        # what no row sees: pages past the first keys' and before the first row's window
        first = (kv - rows + 1 - window) // page
        table = s.table.clone()
        s.table[0, 2:first] = -1
        assert torch.equal(s.run(max_kv=stated, window=window, sinks=sinks), want)
        s.table[0, 2:first] = 2 ** 31 - 1
        assert torch.equal(s.run(max_kv=stated, window=window, sinks=sinks), want)
        # a page of the first keys, or one past the table: all rows, or those that see it
        s.table[0, 1] = s.pages
        got = s.run(max_kv=stated, window=window, sinks=sinks)
        assert bool(torch.isnan(got[:rows]).all()) and torch.equal(got[rows:], want[rows:])
        s.table = table.clone()
        last = (kv - 1) // page
        s.table[0, last] = -7
        got = s.run(max_kv=stated, window=window, sinks=sinks)
        sees = torch.arange(rows) + kv - rows >= last * page
        assert bool(torch.isnan(got[:rows].cpu()[sees]).all())
        assert not bool(torch.isnan(got[:rows].cpu()[~sees]).any())
        s.table = table


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("page,dt", [(16, BF16), (64, F16), (4, BF16)])
@pytest.mark.parametrize("rows,D", [(1, 64), (4, 128), (30, 256), (120, 128), (70, 64)])
def test_odd_values_in_windows(pq, dev, rows, D, page, dt, kind):  # noqa: F811
    """Infinities and NaN in values or keys reach the rows that see them, and no others."""
    kv, window, sinks = rows + 400, 90, 10
    for what in ("value", "key"):
        for sink in (False, True):
            s = kind(pq, dev, [rows], [kv], 1, 2, D, page, dt, seed=3)
            x = s.v[0] if what == "value" else s.k[0]
            x[kv - 1, 0, 5] = float("nan")                  # only the last row sees it
            if what == "value":
                x[kv - max(1, rows // 2), 0, 9] = float("-inf")
            x[sinks + 1, 0, 3] = float("nan")               # no row sees it
            x[kv - rows - window, 0, 40] = float("nan")
            if sink:
                x[sinks - 1, 0, 3] = float("inf")           # every row sees it
            s.fill()
            for out in (dt, F32):
                for stated in STATED:
                    got = s.run(max_kv=stated, window=window, sinks=sinks, out_dtype=out)
                    s.check(got, True, window, sinks, where=f"odd {what}, {sink}, stated {stated}",
                            rows=6)
                    few = got[:max(0, rows - 6)]
                    if what == "value":
                        assert bool(torch.isfinite(few[..., 33:]).all()) or rows < 60


@pytest.mark.parametrize("rows,D", [(1, 64), (4, 128), (30, 256), (120, 128)])
@pytest.mark.parametrize("page", [4, 32])
def test_attention4_any_scale_byte_elsewhere(pq, dev, rows, D, page):  # noqa: F811
    """Bytes the append does not write, as values that only the last row sees: no other
    row's result is touched."""
    kv = rows + 90
    s = Pages4(pq, dev, [rows, 3], [kv, 33], 1, 2, D, page, F16, seed=5)
    p, r = int(s.table[0, (kv - 1) // page]), (kv - 1) % page
    for stated in STATED:
        for byte in (0, 50, 141, 200, 254, 255):
            s.cache.v_scale[p, :, r] = byte
            got = s.run(max_kv=stated)
            base = s.run(max_kv=stated)
            s.cache.v_scale[p, :, r] = 127
            want = s.run(max_kv=stated)
            assert torch.equal(got.nan_to_num(9), base.nan_to_num(9))
            keep = torch.ones(rows + 3, dtype=torch.bool)
            keep[rows - 1] = False
            assert torch.equal(got.cpu()[keep], want.cpu()[keep]), (stated, byte)
            if byte == 255:
                assert bool(torch.isnan(got[rows - 1]).all())


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 3, 90])
def test_attention4_of_the_largest_and_smallest_scales(pq, dev, rows, dt):  # noqa: F811
    """Values at both ends of what a cache holds."""
    lo, hi = ref4.EXPONENTS[dt]
    s = Pages4(pq, dev, [rows], [200 + rows], 1, 2, 64, 16, dt)
    for n in (lo, hi):
        # bf16: as the 16-bit kernels allow, sums of any finite values; their average is finite
        s.v[0] = (s.v[0].double().sign() * 6.0 * 2.0 ** n).to(dt)
        s.v[0][..., ::3] = 2.0 ** n
        s.fill()
        for stated in STATED:
            for out in (dt, F32):
                got = s.run(max_kv=stated, out_dtype=out)
                assert bool(torch.isfinite(got).all())
                e, w, spread = ref4.attention(s.q, s.k[0], s.v[0], 0.125, True, 0, 0)
                # below 2^-111 products lose bits of fp32, as there (2^-129 of one each)
                b = ref.attention_bound(e, w, spread, s.kvs[0], float(s.v[0].double().abs().max()), 64,
                                        dt, out) + 3 * s.kvs[0] * 2.0 ** -129
                check(got, e, b, f"exponent {n}, stated {stated}")


def test_attention4_far_into_a_large_cache(pq, dev):  # noqa: F811
    """Code offsets past 2^32, scales past 2^29."""
    Hk, page, D = 8, 64, 256
    pages = (1 << 32) // (Hk * page * D // 2) + 40
    big = pq.KV4Cache.empty(pages, page, Hk, D, BF16, dev)
    for rows, stated in ((1, 200), (40, 200), (40, 10 ** 6)):
        s = Pages4(pq, dev, [rows], [200], Hk, 2, D, page, BF16)
        far = torch.tensor([pages - 1, 3, pages - 7, pages // 2 + 1])
        for i, p in enumerate(far.tolist()):
            for name in ("k", "k_scale", "v", "v_scale"):
                getattr(big, name)[p] = getattr(s.cache, name)[int(s.table[0, i])]
        s.table[0, :4] = far.to(torch.int32)
        s.cache = big
        s.check(s.run(max_kv=stated), rows=5, where="large cache")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("rows,D,out", [(1, 256, BF16), (3, 64, F32), (40, 128, BF16)])
def test_strides_and_unowned_rows(pq, dev, rows, D, out, kind):  # noqa: F811
    s = kind(pq, dev, [rows, 2], [rows + 177, 9], 2, 3, D, 16, BF16)
    q, cache, table, cu, kv = s.args()
    T = q.shape[0]
    wide = torch.zeros(T + 4, 8 * D * 6, dtype=BF16, device=dev)
    qs = wide[:, D:D + 6 * D].unflatten(1, (6, D))
    qs[2:2 + T] = q
    hold = torch.full((6, T + 4, D + 8), 7.0, dtype=out, device=dev)
    o = hold[:, :, :D].transpose(0, 1)                  # heads outside tokens
    for stated in STATED:
        got = s.call(qs, cache, table, cu + 2, kv, max_q=rows, max_kv=stated, out=o, window=40, sinks=6)
        assert got is o
        s.check(o[2:2 + T], True, 40, 6, where="strided")
    assert bool((hold[:, :2] == 7).all()) and bool((hold[:, T + 2:] == 7).all())
    assert bool((hold[:, :, D:] == 7).all())


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_more_pages_than_a_workgroup_holds(pq, dev, kind):  # noqa: F811
    """Pages of one key, first keys and a window of thousands: the page numbers are
    taken in pieces, with the jump in one of them."""
    s = kind(pq, dev, [20], [13000], 1, 2, 64, 1, BF16)
    for window, sinks in ((5000, 4200), (4090, 10), (9000, 3000)):
        for stated in STATED + [10 ** 9]:
            got = s.run(max_kv=stated, window=window, sinks=sinks)
            s.check(got, True, window, sinks, rows=2, where=f"{window}, {sinks}, stated {stated}")


def test_numbers_past_their_c_types(pq, dev):  # noqa: F811
    for kind in KINDS:
        s = kind(pq, dev, [3], [300], 2, 2, 64, 16, BF16)
        want = s.run(window=50, sinks=300)
        for sinks in (2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 64 + 1):
            assert torch.equal(s.run(window=50, sinks=sinks), want), sinks
        for bad in (dict(window=50, sinks=-1), dict(window=50, sinks=5 - 2 ** 32), dict(sinks=4),
                    dict(causal=False, window=3, sinks=1)):
            with pytest.raises(pq.Pq1Error):
                s.run(**bad)


def test_whole_path_of_a_4_bit_layer_in_a_graph(pq, dev):  # noqa: F811
    """Norms, rotation, append and attention of decoded tokens as they are used
    together, captured; each replay reads the present inputs, with eager work in
    between, and a prompt went in before by the same calls in chunks."""
    Hk, G, D, page, B = 2, 4, 128, 16, 2
    w = (1 + 0.2 * torch.randn(2, D, generator=torch.Generator().manual_seed(1))).to(dev)
    norm = pq.HeadNorm(w[0], w[1], eps=1e-6)
    rope = pq.Rope(64, freqs=pq.rope_frequencies(64, device=dev))
    table = torch.randperm(80, generator=torch.Generator().manual_seed(2)).view(B, 40).to(torch.int32)
    cu = lambda n: torch.tensor([0, n, 2 * n], dtype=torch.int32, device=dev)
    gt = table.to(dev)

    def call(cache, x, at, q0, n):
        """x [B n][heads][D] at positions at [B n]; lens [B]."""
        slots = gt[torch.arange(B, device=dev).repeat_interleave(n), at // page].long() * page + at % page
        q = pq.pq1_kv4_append(cache, x[:, :Hk], x[:, Hk:2 * Hk], slots, positions=at.to(torch.int32),
                              rope=rope, q=x[:, 2 * Hk:], norm=norm)
        lens = at.view(B, n)[:, -1].to(torch.int32) + 1
        return q, pq.pq1_kv4_attention(q, cache, gt, q0, lens, max_q=n, max_kv=600, window=150, sinks=4,
                                       out_dtype=F32)

    def fresh():
        cache = pq.KV4Cache.empty(80, page, Hk, D, BF16, dev)
        g = torch.Generator(device=dev).manual_seed(3)
        for start, n in ((0, 300), (300, 20)):
            x = torch.randn(B * n, (2 + G) * Hk, D, device=dev, generator=g)
            at = (torch.arange(n, device=dev) + start).repeat(B)
            call(cache, x, at, cu(n), n)
        return cache

    cache, twin = fresh(), fresh()
    x = torch.zeros(B, (2 + G) * Hk, D, device=dev)
    at = torch.tensor([320, 320], device=dev)
    one = cu(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(fresh(), x, at, one, 1)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q_out, out = call(cache, x, at, one, 1)
    for turn in range(5):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(turn)))
        at.fill_(320 + turn)
        graph.replay()
        want_q, want = call(twin, x, at, one, 1)
        torch.cuda.synchronize()
        assert torch.equal(q_out, want_q) and torch.equal(out, want), f"replay {turn}"
    # against the formulas, from what the cache holds
    slots = torch.cat([gt[b].long().repeat_interleave(page) * page + torch.arange(640, device=dev) % page
                       for b in range(B)])
    k, v = (t.cpu().view(B, 640, Hk, D)[:, :325] for t in pq.pq1_kv4_read(twin, slots))
    for b in range(B):
        e, wt, spread = ref4.attention(q_out[b:b + 1].cpu(), k[b], v[b], D ** -0.5, True, 150, 4)
        check(out[b:b + 1], e, ref.attention_bound(e, wt, spread, 325, 0.0, D, BF16, F32), "layer")


def test_graphs_of_one_capture_stream_replayed_on_two(pq, dev):  # noqa: F811
    """Calls of parts (a workspace each): graphs replayed at the same time on two
    streams, with calls of their own on a third."""
    batches = [Pages4(pq, dev, [1], [9000 + 100 * i], 1, 6, 256, 64, BF16, seed=i) for i in range(3)]
    args = [b.args() for b in batches]
    call = lambda i: pq.pq1_kv4_attention(*args[i], max_q=1, max_kv=9000 + 100 * i)
    assert pq.load_library().pq1_kv4_attention_workspace_bytes(1, 1, 6, 1, 256, 1, 9000, 0, 0) > 0
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


def stretched(s, tile_rows, max_q, max_kv, window=0, sinks=0):
    """That such a call cuts the batch's work evenly among workgroups: its workspace is
    two slots of a row tile for each and a note for every row tile."""
    lib = s.pq.load_library()
    fn = (lib.pq1_kv4_attention_workspace_bytes if isinstance(s, Pages4) else
          lib.pq1_paged_attention_ex_workspace_bytes)
    B, T, Hq = len(s.qs), s.q.shape[0], s.Hk * s.G
    got = fn(B, T, Hq, s.Hk, s.D, max_q, max_kv, window, sinks)
    notes = 8 * s.Hk * (T * s.G // tile_rows + B + 1)
    return got in [2 * wgs * tile_rows * (4 * s.D + 8) + notes for wgs in (256, 512)]


STRETCHES = [
    # new tokens, keys, Hk, G, D, page, type, out
    ([1, 1], [1500, 1], 1, 1, 128, 16, BF16, BF16),                  # fewer steps than workgroups
    ([1] * 40, [1 + 37 * i for i in range(40)], 4, 6, 256, 64, BF16, BF16),
    ([1] * 40, [1400 - 35 * i for i in range(40)], 4, 6, 128, 8, F16, F32),
    ([1, 0, 1, 0, 0, 1], [900, 70, 0, 0, 3, 2000], 3, 2, 128, 32, F16, F16),
    ([4, 1, 0, 6, 2], [700, 2, 5, 300, 1300], 2, 4, 256, 16, BF16, F32),
    ([40, 3, 17], [900, 3, 650], 2, 5, 128, 16, BF16, BF16),         # more tokens than was said
    ([1] * 130, [(i * 41) % 160 for i in range(130)], 1, 8, 256, 4, F16, F16),
    ([2] * 3 + [0] * 70 + [3] * 3, [500] * 3 + [9] * 70 + [800] * 3, 2, 2, 128, 16, BF16, BF16),
]


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("case", STRETCHES, ids=range(len(STRETCHES)))
def test_work_cut_evenly(pq, dev, case, kind):  # noqa: F811
    """Batches whose work is cut into stretches, whatever tiles these begin and end in:
    all keys, and first keys before a window that leaves none out or nearly all."""
    qs, kvs, Hk, G, D, page, dt, dout = case
    s = kind(pq, dev, qs, kvs, Hk, G, D, page, dt, seed=len(qs))
    max_q = min(max(qs), 32 // G)
    tile_rows = 16 if max_q * G <= 16 else 32
    for window, sinks in ((0, 0), (10 ** 8, 7), (90, 10 ** 8)):
        if window == 0 and kind is Pages:
            continue                        # the plain kernel's
        assert stretched(s, tile_rows, max_q, 2 ** 31, window, sinks), (window, sinks)
        got = s.run(max_q=max_q, max_kv=2 ** 31, window=window, sinks=sinks, out_dtype=dout)
        s.check(got, True, window, sinks, where=f"window {window}")
        again = s.run(max_q=max_q, max_kv=2 ** 31, window=window, sinks=sinks, out_dtype=dout)
        assert torch.equal(got, again), "the same call gives the same bits"


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_odd_values_in_work_cut_evenly(pq, dev, kind):  # noqa: F811
    """Infinities and NaN in values that only the last of a sequence's rows sees, in tiles
    that several workgroups have parts of."""
    qs, kvs = [3, 1, 5, 2], [2000, 900, 1400, 40]
    s = kind(pq, dev, qs, kvs, 2, 3, 128, 16, BF16, seed=4)
    for b, n in enumerate(kvs):
        s.v[b][n - 1, 0, 5] = float("nan")
        s.v[b][n - 1, 1, 77] = float("-inf")
    s.fill()
    assert stretched(s, 16, 5, 2 ** 31, 10 ** 8, 4)
    for out in (BF16, F32):
        got = s.run(max_q=5, max_kv=2 ** 31, window=10 ** 8, sinks=4, out_dtype=out)
        s.check(got, True, 10 ** 8, 4, where="odd values")


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
def test_work_cut_evenly_in_graphs(pq, dev, kind):  # noqa: F811
    """A captured call cuts by the lengths of its replay; two graphs and an eager call at
    once, each with its own workspace."""
    sizes = [([1, 1, 1], [700, 1500, 90]), ([2, 1, 4], [800, 20, 1100]), ([1, 1, 1], [64, 900, 300])]
    batches = [kind(pq, dev, qs, kvs, 4, 6, 256, 64, BF16, seed=i) for i, (qs, kvs) in enumerate(sizes)]
    args = [b.args() for b in batches]
    kw = dict(max_q=4, max_kv=2 ** 31, window=10 ** 8, sinks=5)
    call = lambda i: batches[i].call(*args[i], **kw)
    assert all(stretched(b, 32, 4, 2 ** 31, 10 ** 8, 5) for b in batches)
    want = [call(i).clone() for i in range(3)]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(i))
        graphs.append(g)
    for turn in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(10):
            for i in range(2):
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
            third = call(2)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i]), f"graph {i}, turn {turn}"
        assert torch.equal(third, want[2])
    # other lengths in the same tensors
    kv = args[0][4]
    for lens in ([1, 1400, 33], [700, 3, 0], [640, 1500, 90]):
        kv.copy_(torch.tensor(lens, dtype=torch.int32))
        graphs[0].replay()
        got = outs[0].clone()
        assert torch.equal(got, call(0)), lens
        for b, n in enumerate(lens):
            e, w, spread = ref4.attention(batches[0].q[b:b + 1], batches[0].k[b][:n],
                                          batches[0].v[b][:n], 1 / 16, True, 0, 0)
            check(got[b:b + 1], e, ref.attention_bound(
                e, w, spread, n, float(batches[0].v[b].double().abs().max()), 256, BF16, BF16),
                f"lengths {lens}, sequence {b}")


@pytest.mark.parametrize("bits", [16, 4])
def test_attention_layer_example(pq, dev, bits):  # noqa: F811
    """The example's layer with norms and a window with first keys: in chunks and single
    tokens it runs, and its attention is the formula's over what its cache holds."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                    "examples"))
    import attention_layer as ex
    layer = ex.AttentionLayer(hidden=1024, heads=4, kv_heads=2, dim=256, pages=40, page_size=16,
                              norms=True, bits=bits, window=40, sinks=3)
    x = torch.randn(150, 1024, device=dev, generator=torch.Generator(device=dev).manual_seed(1))
    parts = ex.run(layer, x, range(30, 20, -1), [64, 1, 50, 33, 1, 1])
    assert parts.shape == x.shape and bool(torch.isfinite(parts).all())
    whole = ex.run(layer, x, range(10), [150])
    D, a = 256, ex.Sequence(layer, range(10)).extend(150)
    qkv = layer._project(x, layer.qkv)
    q, k, v = (qkv[:, i * D:j * D].unflatten(1, (j - i, D)) for i, j in ((0, 4), (4, 6), (6, 8)))
    qr = layer.append(layer.cache, k, v, a["slots"], positions=a["positions"], rope=layer.rope, q=q,
                      norm=layer.norm)
    o = layer.attend(qr, layer.cache, a["table"], a["cu_q"], a["kv_len"], 150, 150, window=40, sinks=3,
                     out_dtype=F32)
    assert torch.equal(layer._project(o.view(150, 4 * D), layer.out), whole)
    if bits == 4:
        kc, vc = pq.pq1_kv4_read(layer.cache, a["slots"])
    else:
        kc, vc = (t[:10].transpose(1, 2).reshape(160, 2, D)[:150] for t in (layer.cache.k, layer.cache.v))
    e, w, spread = ref4.attention(qr.cpu(), kc.cpu(), vc.cpu(), D ** -0.5, True, 40, 3)
    check(o, e, ref.attention_bound(e, w, spread, 150, float(vc.double().abs().max()), D, BF16, F32),
          "example")
