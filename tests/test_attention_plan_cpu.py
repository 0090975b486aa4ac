"""How an attention call is cut (csrc/attn_plan.h), checked on the host: the
parts that the kernels write always fit the workspace that the size call asks
for, whatever the caller states as its longest chunk and cache."""
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_hadamard_rotated_amd", "csrc")
MAX_KEYS = 0x7fff0000

PROGRAM = """
#include <stdio.h>
#include "attn_plan.h"
int main() {
  long long B, T, Hq, Hk, D, mq, mkv, w;
  while (scanf("%lld %lld %lld %lld %lld %lld %lld %lld", &B, &T, &Hq, &Hk, &D, &mq, &mkv, &w) == 8) {
    const pq1::AttnPlan size = pq1::plan_attention(B, T, Hq, Hk, D, mq, mkv);
    const pq1::AttnPlan p = pq1::plan_attention(B, T, Hq, Hk, D, mq, mkv, w);
    printf("%d %d %d %lld %d %d %zu %zu\\n", p.fits, p.many, p.tile_rows,
           static_cast<long long>(p.row_tiles), p.nsplit, p.chunk, p.workspace_bytes,
           size.workspace_bytes);
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


def check_plan(sizes, plan):
    B, T, Hq, Hk, D, mq, mkv, w = sizes
    fits, many, tile_rows, row_tiles, nsplit, chunk, ws, ws_of_size_call = plan
    if not fits:
        return
    assert nsplit >= 1 and chunk >= 128 and chunk % 128 == 0 and row_tiles >= 1, sizes
    parts = nsplit * T * Hq * (4 * D + 8) if nsplit > 1 else 0
    assert ws >= parts, f"{sizes}: {nsplit} parts in {ws} bytes"
    assert ws == ws_of_size_call, sizes       # the size call knows no window
    # the parts cover the keys stated
    keys = min(max(mkv, 1), MAX_KEYS)
    if w:
        keys = min(keys, w + tile_rows + 64)
    assert nsplit * chunk >= keys, sizes
    assert chunk <= MAX_KEYS + 128 and chunk < 2 ** 31, sizes
    assert B * Hk * row_tiles * nsplit * (512 if many else 256) < 2 ** 32, sizes


FAR = [1, 700, 2 ** 20, MAX_KEYS - 1, MAX_KEYS, MAX_KEYS + 1, 0x7fffff00, 0x7fffff01, 2 ** 31 - 1,
       2 ** 31, 2 ** 40, 2 ** 62]


@pytest.mark.parametrize("B,T,Hq,Hk,D,mq", [
    (64, 64, 24, 4, 256, 1),           # decoding users that fill the device
    (1, 4000, 24, 4, 256, 4000),       # a prompt that does
    (1, 1, 8, 1, 64, 1), (1, 2048, 24, 4, 256, 2048), (300, 300, 8, 1, 128, 1),
    (5, 20000, 32, 8, 128, 4000), (2, 2, 2, 2, 64, 1)])
def test_parts_fit_the_workspace_at_any_stated_length(plans, B, T, Hq, Hk, D, mq):
    sizes = [(B, T, Hq, Hk, D, mq, mkv, w) for mkv in FAR
             for w in (0, 1, 1024, 2 ** 30, 2 ** 31 - 1)]
    for s, p in zip(sizes, plans(sizes)):
        check_plan(s, p)


def test_parts_fit_the_workspace_at_any_sizes(plans):
    rng = random.Random(5)
    log = lambda hi: int(2 ** rng.uniform(0, hi))
    sizes = []
    for _ in range(20000):
        Hk = log(10)
        G = rng.randint(1, max(1, min(64, 1024 // Hk)))
        T = min(log(30), 0x7ff00000 // (Hk * G))
        sizes.append((log(23), T, Hk * G, Hk, rng.choice([64, 128, 256]), log(62),
                      rng.choice([log(62), log(32), rng.choice(FAR)]),
                      rng.choice([0, 0, min(log(31), 2 ** 31 - 1)])))
    for s, p in zip(sizes, plans(sizes)):
        check_plan(s, p)
