"""How an attention call whose workspace knows its window is cut (plan_window of
csrc/attn_plan.h), checked on the host, and what those calls refuse."""
import math
import os
import random
import shutil
import subprocess

import pytest

from conftest import gpu_available
from gemm_hadamard_rotated_amd import pq1
from test_attention_abi_cpu import (ALIAS, ALIGN, ARG, BF16, BIG, F16, F32, GIB, NULL, OK, P, SHAPE,
                                    cache, heads, lib)  # noqa: F401 (lib: a fixture)
from test_kv4_abi_cpu import DEVICE, cache4

needs_no_gpu = pytest.mark.skipif(gpu_available(), reason="needs a host without a visible GPU")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_hadamard_rotated_amd", "csrc")
MAX_KEYS = 0x7fff0000
FORMS = ("0", "1")          # caches of two-byte and of 4-bit numbers

PROGRAM = """
#include <stdio.h>
#include "attn_plan.h"
int main() {
  long long B, T, Hq, Hk, D, mq, mkv, w, s, four;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld %lld %lld", &B, &T, &Hq, &Hk, &D, &mq, &mkv, &w,
               &s, &four) == 10) {
    const pq1::AttnPlan p = pq1::plan_window(B, T, Hq, Hk, D, mq, mkv, w, s, four != 0);
    printf("%d %d %d %lld %d %d %zu %d %d\\n", p.fits, p.many, p.tile_rows,
           static_cast<long long>(p.row_tiles), p.nsplit, p.chunk, p.workspace_bytes, p.wgs,
           p.joined);
  }
}
"""


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    cc = next((c for c in (shutil.which("g++"), shutil.which("c++"), shutil.which("clang++")) if c),
              None)
    if cc is None:
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("plan")
    (at / "plan.cpp").write_text(PROGRAM)
    subprocess.run([cc, "-std=c++17", "-O1", f"-I{CSRC}", "-o", str(at / "plan"),
                    str(at / "plan.cpp")], check=True)

    def run(sizes):
        text = "\n".join(" ".join(str(n) for n in s) for s in sizes)
        out = subprocess.run([str(at / "plan")], input=text, stdout=subprocess.PIPE, text=True,
                             check=True).stdout
        rows = [tuple(int(n) for n in line.split()) for line in out.splitlines()]
        assert len(rows) == len(sizes)
        return rows

    return run


def walked(row0, rows, G, n, kv, w, s, tile):
    """Keys that a tile of these rows walks over, as the kernels do: the first keys
    rounded up to key tiles, then the window from its start rounded down to them."""
    i0, i1 = row0 // G, min(row0 + rows - 1, n * G - 1) // G
    end = max(0, kv - (n - 1 - i1))
    lo = max(0, kv - (n - 1 - i0) - w) if w else 0
    first, sink_end = lo // tile * tile, -(-s // tile) * tile
    return end - max(0, first - sink_end)


def test_parts_cover_what_tiles_walk_over(plans):
    rng = random.Random(3)
    log = lambda hi: int(2 ** rng.uniform(0, hi))
    sizes = []
    for _ in range(20000):
        Hk = log(10)
        G = rng.randint(1, max(1, min(64, 1024 // Hk)))
        T = min(log(30), 0x7ff00000 // (Hk * G))
        w = rng.choice([0, min(log(31), 2 ** 31 - 1), log(12)])
        sizes.append((log(23), T, Hk * G, Hk, rng.choice([64, 128, 256]), log(rng.choice([3, 62])),
                      rng.choice([log(62), log(20), MAX_KEYS, 2 ** 62]), w,
                      rng.choice([0, 4, min(log(31), 2 ** 31 - 1)]) if w else 0, rng.randint(0, 1)))
    for size, plan in zip(sizes, plans(sizes)):
        B, T, Hq, Hk, D, mq, mkv, w, s, four = size
        fits, many, tile_rows, row_tiles, nsplit, chunk, ws, wgs, joined = plan
        if not fits:
            continue
        assert row_tiles >= 1 and nsplit >= 1, size
        assert B * Hk * row_tiles * nsplit * (512 if many else 256) < 2 ** 32, size
        n, kv, G = min(max(mq, 1), T), min(max(mkv, 1), MAX_KEYS), Hq // Hk
        if not many:
            # the rows of each part; or two slots for each stretch, and a note for every
            # row tile there may be
            assert tile_rows in (16, 32) and wgs <= 768 and (nsplit == 1 or wgs == 0), size
            tiles = T * G // tile_rows + B + 1
            parts = nsplit * T * Hq * (4 * D + 8) if nsplit > 1 else 0
            assert ws == (2 * wgs * tile_rows * (4 * D + 8) + 8 * tiles * Hk if wgs else parts), size
            assert joined == (wgs > 0 or nsplit > 1), size
            continue
        assert wgs == 0 and joined == (nsplit > 1), size
        assert chunk >= 128 and chunk % 128 == 0, size
        assert ws == (nsplit * T * Hq * (4 * D + 8) if nsplit > 1 else 0), size
        assert chunk <= MAX_KEYS + 128 and chunk < 2 ** 31, size
        # what a stated chunk's tiles walk over fits the parts without stretching them
        for row0 in (0, tile_rows, (n * G - 1) // tile_rows * tile_rows):
            if row0 < n * G:
                assert walked(row0, tile_rows, G, n, kv, w, s, 32 if D == 256 else 64) <= nsplit * chunk, size


def test_a_window_that_hides_no_key_is_cut_as_none(plans):
    """And one that is short beside the longest sequence leaves the tiles of a large
    batch whole."""
    rng = random.Random(5)
    sizes = [(64, 64, 24, 4, 256, 1, 8000, w, s, four) for w in (8000, 10 ** 6) for s in (0, 16)
             for four in (0, 1)]
    for _ in range(3000):
        Hk, mkv = rng.choice([1, 2, 4, 8]), int(2 ** rng.uniform(0, 18))
        B, n = rng.randint(1, 600), rng.choice([1, 1, 2, 6, 40])
        sizes.append((B, B * n, Hk * rng.randint(1, 8), Hk, rng.choice([64, 128, 256]), n, mkv,
                      mkv + rng.randint(0, 1000), rng.choice([0, 4, 100]), rng.randint(0, 1)))
    none = [(*s[:7], 0, 0, s[9]) for s in sizes]
    for size, got, want in zip(sizes, plans(sizes), plans(none)):
        assert got == want, size
    for four in (0, 1):
        assert plans([(64, 64, 24, 4, 256, 1, 8000, 0, 0, four)])[0][7] > 0
        whole = plans([(64, 64, 24, 4, 256, 1, 8000, 1024, 4, four),
                       (48, 48, 32, 8, 128, 1, 30000, 1024, 4, four)])
        assert all(p[4] == 1 and p[7] == 0 and not p[8] for p in whole)


def test_notes_of_row_tiles_do_not_meet():
    """Where the kernels note a tile's pieces: q0 G / ROWS + b on, for sequences that
    follow one another; and never past the workspace, whatever cu_q holds."""
    rng = random.Random(1)
    for _ in range(2000):
        G, rows = rng.randint(1, 40), rng.choice([16, 32])
        lens = [rng.choice([0, 1, rng.randint(0, 60)]) for _ in range(rng.randint(1, 12))]
        q0, last = 0, -1
        for b, n in enumerate(lens):
            first, tiles = q0 * G // rows + b, -(-n * G // rows)
            assert first > last, (G, rows, lens)
            last = max(last, first + tiles - 1)
            q0 += n
        assert last < q0 * G // rows + len(lens) + 1
        T, B = q0, len(lens)
        for b in range(B):                       # any two numbers within [0, T]
            a, z = sorted((rng.randint(0, T), rng.randint(0, T)))
            assert a * G // rows + b + -(-(z - a) * G // rows) <= T * G // rows + B + 1


def attend(lib, fn, q=None, out=None, c=None, table=P(3 * GIB), max_pages=100, cu=P(4 * GIB),  # noqa: F811
           kv=P(5 * GIB), B=2, T=4, Hq=16, max_q=2, max_kv=90, scale=0.1, causal=1, window=64, sinks=4,
           ws=P(8 * GIB), wsb=1 << 30):
    c = (cache() if fn == "pq1_paged_attention_ex" else cache4()) if c is None else c
    return getattr(lib, fn)(heads(GIB, n=16) if q is None else q,
                            heads(2 * GIB, n=16) if out is None else out, c, table, max_pages, cu, kv, B,
                            T, Hq, max_q, max_kv, scale, causal, window, sinks, ws, wsb, None)


@pytest.mark.parametrize("fn", ["pq1_paged_attention_ex", "pq1_kv4_attention"])
def test_refusals(lib, fn):  # noqa: F811
    a = lambda **kw: attend(lib, fn, **kw)
    make = cache if fn == "pq1_paged_attention_ex" else cache4
    call = getattr(lib, fn)
    rest = (P(8), 1, P(8), P(8), 1, 1, 8, 1, 1, 0.1, 1, 0, 0, None, 0, None)
    assert call(None, heads(GIB), make(), *rest) == NULL
    assert call(heads(GIB), None, make(), *rest) == NULL
    assert call(heads(GIB), heads(GIB), None, *rest) == NULL
    assert a(table=None) == NULL and a(cu=None) == NULL and a(kv=None) == NULL
    assert a(q=heads(None, n=16)) == NULL and a(c=make(v=None)) == NULL
    assert a(q=heads(GIB, F16, n=16)) == ARG and a(out=heads(2 * GIB, F16, n=16)) == ARG
    assert a(c=make(dtype=F32)) == ARG
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert a(scale=scale) == ARG
    assert a(causal=2) == ARG and a(window=-1) == ARG and a(causal=0) == ARG
    assert a(sinks=-1) == ARG and a(sinks=-(1 << 31)) == ARG
    assert a(sinks=1, window=0) == ARG and a(causal=0, window=0, sinks=3) == ARG
    for bad in (dict(Hq=15), dict(Hq=4), dict(Hq=1032), dict(B=-1), dict(T=-1), dict(max_q=-1),
                dict(max_kv=-1), dict(max_pages=-1), dict(max_pages=1 << 31), dict(T=1 << 30),
                dict(c=make(D=96)), dict(c=make(page=3))):
        assert a(**bad) == SHAPE, bad
    assert a(q=heads(GIB + 8, n=16)) == ALIGN and a(cu=P(4 * GIB + 2)) == ALIGN
    arrays = (BIG, 2 * BIG) if fn == "pq1_paged_attention_ex" else (BIG, 2 * BIG, 3 * BIG, 4 * BIG)
    for at in (GIB, 3 * GIB, 4 * GIB, 5 * GIB, *arrays):
        assert a(out=heads(at, n=16)) == ALIAS
    # a workspace is needed where the keys are cut into parts
    size = getattr(lib, fn + "_workspace_bytes")
    far = dict(max_kv=100000, max_pages=10000, window=50000)
    need = size(2, 4, 16, 8, 128, 2, 100000, 50000, 4)
    assert need > 0
    assert a(ws=None, **far) == NULL and a(ws=P(8 * GIB + 128), **far) == ALIGN
    assert a(wsb=need - 1, **far) == ARG
    for at in (GIB, 2 * GIB, *arrays):
        assert a(ws=P(at), **far) == ALIAS
    assert a(B=0) == OK and a(T=0) == OK
    for bad in ((2, 4, 15, 8, 128, 2, 9, 0, 0), (2, 4, 16, 8, 80, 2, 9, 0, 0), (2, 4, 16, 8, 128, 2, 9, -1, 0),
                (2, 4, 16, 8, 128, 2, 9, 5, -1), (2, 4, 16, 8, 128, 2, 9, 0, 5), (0, 4, 16, 8, 128, 2, 9, 0, 0)):
        assert size(*bad) == 0


@needs_no_gpu
@pytest.mark.parametrize("fn", ["pq1_paged_attention_ex", "pq1_kv4_attention"])
def test_accepted_up_to_the_device_check(lib, fn):  # noqa: F811
    a = lambda **kw: attend(lib, fn, **kw)
    assert a() == DEVICE and a(ws=None, wsb=0) == DEVICE and a(sinks=0) == DEVICE
    assert a(window=0, sinks=0, causal=0) == DEVICE and a(table=None, max_pages=0) == DEVICE
    assert a(out=heads(2 * GIB, F32, n=16)) == DEVICE
    top = (1 << 31) - 1
    need = getattr(lib, fn + "_workspace_bytes")(2, 4, 16, 8, 128, 2, 1 << 62, top, top)
    assert a(window=top, sinks=top, max_kv=1 << 62, wsb=need) == DEVICE


def test_binding_refusals():
    with pytest.raises(TypeError, match="KV4Cache"):
        pq1.pq1_kv4_attention(None, None, None, None, None, 1, 1)
