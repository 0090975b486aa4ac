"""The few-rows attention kernel over 4-bit caches keeps V's loads in flight over the
products of K, checked on the gfx950 assembly that the compiler makes (no GPU).

A tile's turn issues the loads of V (codes and scales of eight keys, 16 loads) and then
takes the products of K, which were loaded a tile earlier.  Where V's scales are touched
ahead of those products, each tile waits for memory twice (15 % of a decode in a window)."""
import os
import re
import shutil
import subprocess

import pytest

from test_attention_isa_cpu import CSRC

LOADS = 16  # of V, by a lane


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    cc = next((c for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc"))
               if c and os.path.exists(c)), None)
    if cc is None:
        pytest.skip("hipcc not available")
    from gemm_hadamard_rotated_amd import build
    out = tmp_path_factory.mktemp("isa") / "few.s"
    source = "kv4_attention.hip"
    flags = [f for f in build.flags_for(source) if f != "-fPIC"]
    p = subprocess.run([cc, *flags, "--cuda-device-only", "-S", "-o", str(out),
                        os.path.join(CSRC, source)],
                       stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0, p.stdout[-4000:]
    # pages of 16 keys or more, heads of 128 and 256
    return re.findall(r"^(_ZN\w*few_stretch_kernel\w+Li(?:128|256)ELi[12]ELb1E\w+):[^\n]*\n(.*?)"
                      r"\.end_amdhsa_kernel", out.read_text(), re.S | re.M)


def test_products_of_k_do_not_wait_for_v(kernels):
    assert len(kernels) == 16
    for name, body in kernels:
        lines = [l.strip() for l in body.splitlines()]
        product = next(i for i, l in enumerate(lines) if l.startswith("v_mfma"))
        loads = [i for i in range(product) if lines[i].startswith("buffer_load")]
        waits = [int(m.group(1)) for l in lines[loads[-1]:product]
                 if (m := re.search(r"s_waitcnt .*vmcnt\((\d+)\)", l))]
        # for K, and none that leaves less than V's loads in flight
        assert waits and min(waits) >= LOADS, f"{name}: {waits}"
