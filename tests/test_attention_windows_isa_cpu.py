"""The order of copies and waits in the many-rows kernel of windows whose first keys
stay visible, which walks two runs of keys: what holds for the plain kernel, on the
gfx950 assembly that the compiler makes (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

from test_attention_isa_cpu import CSRC


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    cc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc"))
               if c and os.path.exists(c)), None)
    if cc is None:
        pytest.skip("hipcc not available")
    from gemm_hadamard_rotated_amd import build
    out = tmp_path_factory.mktemp("isa") / "tiles.s"
    source = "paged_attention_tiles_sinks.hip"
    flags = [f for f in build.flags_for(source) if f != "-fPIC"]
    p = subprocess.run([cc, *flags, "--cuda-device-only", "-S", "-o", str(out),
                        os.path.join(CSRC, source)],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0, p.stdout[-4000:]
    return re.findall(r"^(_ZN\w*many_rows_kernel\w+):[^\n]*\n(.*?)\.end_amdhsa_kernel",
                      out.read_text(), re.S | re.M)


def shortest_turn(lines, start):
    """Instructions of the shortest way from one back to itself."""
    label = {m.group(1): i for i, l in enumerate(lines) if (m := re.match(r"(\.LBB\w+):", l))}
    came, todo = {}, [start]
    while todo:
        nxt = []
        for i in todo:
            m = re.match(r"s_(c?)branch\w* (\.LBB\w+)", lines[i])
            to = [label[m.group(2)]] if m else []
            if not (m and not m.group(1)) and not lines[i].startswith("s_endpgm"):
                to.append(i + 1)
            for j in to:
                if j not in came and j < len(lines):
                    came[j] = i
                    nxt.append(j)
        if start in came:
            break
        todo = nxt
    turn, i = {start}, came[start]
    while i != start:
        turn.add(i)
        i = came[i]
    return turn


def test_waits_leave_one_tile_of_copies_in_flight(kernels):
    assert len(kernels) == 24
    for name, body in kernels:
        copies = 2 if "Li64E" in name else 4     # of K and V, by a wave, for a tile
        lines = [l.strip() for l in body.splitlines()]
        copy = [i for i, l in enumerate(lines) if l.startswith("global_load_lds_dwordx4")]
        wait = {i: int(re.search(r"\d+", l).group()) for i, l in enumerate(lines)
                if re.match(r"s_waitcnt vmcnt\(\d+\)$", l) and lines[i - 1] == ";;#ASMSTART"}
        # two tiles before the loop, one in it
        assert len(copy) == 3 * copies, name
        assert sorted(wait.values()) == [0, copies, copies], name
        for i in (i for i, n in wait.items() if n == copies):
            # each ends at a barrier, nothing loaded between
            b = next(j for j in range(i, len(lines)) if lines[j] == "s_barrier")
            between = [l for l in lines[i + 1:b] if re.match(r"(global|buffer|flat|scratch)_", l)]
            assert not between, f"{name}: {between}"
        turns = [shortest_turn(lines, i) for i, n in wait.items() if n == copies]
        turn = min((t for t in turns if any("v_mfma" in lines[i] for i in t)), key=len)
        assert sum(i in turn for i in copy) == copies and sum(i in turn for i in wait) == 1, name
        drains = [lines[i] for i in turn if re.match(r"s_waitcnt .*vmcnt\(0\)", lines[i])]
        assert not drains, f"{name}: {drains}"
