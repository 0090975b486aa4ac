"""The Python side of the attention-layer calls without a GPU: what it passes
on, keeps and refuses, with the library replaced by a recorder."""
import os
import subprocess
import sys

import pytest
import torch

from gemm_hadamard_rotated_amd import pq1

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_module_imports_on_a_torch_without_gpu_support():
    """Such a torch lacks the accessors of the current stream and device; the
    calls then raise for tensors that are not on a GPU."""
    code = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
from gemm_hadamard_rotated_amd import pq1
try:
    pq1.pq1_rope(torch.zeros(2, 4, 64), torch.zeros(1, 2, dtype=torch.int32), None)
except ValueError as e:
    assert "GPU" in str(e)
    print("raised")
"""
    p = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE,
                       stderr=subprocess.STDOUT, text=True)
    assert p.returncode == 0 and "raised" in p.stdout, p.stdout


def test_hints_and_window_of_any_size():
    f = pq1._hints_and_window
    assert f(1, 700, 0) == (1, 700, 0) and f(0, 0, 2 ** 31 - 1) == (0, 0, 2 ** 31 - 1)
    assert f(-1, -1, -1) == (-1, -1, -1)
    for n in (2 ** 31, 2 ** 32, 2 ** 32 + 5, 2 ** 64 + 5):
        assert f(1, 1, n) == (1, 1, 2 ** 31 - 1)
    for n in (2 ** 62, 2 ** 63, 2 ** 64 + 5):
        assert f(n, 3, 0) == (2 ** 62, 3, 0) and f(3, n, 0) == (3, 2 ** 62, 0)
    for n in (-2 ** 31 - 1, -2 ** 32 + 5, -2 ** 64 + 5):
        q, kv, w = f(n, n, n)
        assert q < 0 and kv < 0 and w == -1
