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
