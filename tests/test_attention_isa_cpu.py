"""Order of the copies into LDS in the many-rows attention kernel, checked on
the gfx950 assembly the compiler produces (no GPU).

A tile issues n copies (the tile after next) and ends with a wait until at most
n vector-memory operations are in flight and a barrier: then the copies of the
next tile, issued a tile earlier, have landed.  That holds as long as exactly
the last n copies are younger than the ones waited for, that is if the loop
issues n copies between two such waits.  The waits and copies are written as
instructions, so the compiler knows nothing of them; if it waited for all
vector memory inside the loop on its own account, the copies would be no longer
ahead of the products (this cost 8 % where it happened)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_hadamard_rotated_amd", "csrc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    cc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc"))
               if c and os.path.exists(c)), None)
    if cc is None:
        pytest.skip("hipcc not available")
    from gemm_hadamard_rotated_amd import build
    out = tmp_path_factory.mktemp("isa") / "tiles.s"
    flags = [f for f in build.flags_for("paged_attention_tiles.hip") if f != "-fPIC"]
    p = subprocess.run([cc, *flags, "--cuda-device-only", "-S", "-o", str(out),
                        os.path.join(CSRC, "paged_attention_tiles.hip")],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0, p.stdout[-4000:]
    return re.findall(r"^(_ZN\w*many_rows_kernel\w+):[^\n]*\n(.*?)\.end_amdhsa_kernel",
                      out.read_text(), re.S | re.M)


def test_waits_leave_one_tile_of_copies_in_flight(kernels):
    assert len(kernels) == 24
    for name, body in kernels:
        copies = 2 if "Li64E" in name else 4     # of K and V, by a wave, for a tile
        lines = [l.strip() for l in body.splitlines()]
        copy = [i for i, l in enumerate(lines) if l.startswith("global_load_lds_dwordx4")]
        wait = [i for i, l in enumerate(lines) if re.match(r"s_waitcnt vmcnt\(\d+\)$", l)
                and lines[i - 1] == ";;#ASMSTART"]
        # two tiles before the loop, one in it
        assert len(copy) == 3 * copies, name
        counts = [int(re.search(r"\d+", lines[i]).group()) for i in wait]
        assert sorted(counts) == [0, copies, copies], f"{name}: {counts}"
        ahead = [i for i, n in zip(wait, counts) if n == copies]
        for i in ahead:                          # each ends at a barrier, nothing loaded between
            b = next(j for j in range(i, len(lines)) if lines[j] == "s_barrier")
            between = [l for l in lines[i + 1:b] if re.match(r"(global|buffer|flat|scratch)_", l)]
            assert not between, f"{name}: {between}"
        # No other wait for all vector memory from there to the one after the
        # loop, except before the loop's first block (for the rows of Q).
        label = next(i for i in range(ahead[0], len(lines)) if lines[i].startswith(".LBB"))
        after = wait[counts.index(0)]
        assert ahead[1] < after and copy[-1] < after and label < min(ahead[1], copy[-1]), name
        drains = [lines[i] for i in range(label, after) if i != after
                  and re.match(r"s_waitcnt .*vmcnt\(0\)", lines[i])]
        assert not drains, f"{name}: {drains}"
