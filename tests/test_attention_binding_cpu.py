"""The Python side of the attention-layer calls without a GPU: what it passes
on, keeps and refuses, with the library replaced by a recorder."""
import os
import subprocess
import sys
import threading
import time
import types

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


class Recorder:
    """Stands for the library: a call needs `need` bytes, takes a while, and
    notes the workspaces it was given and the calls that overlapped."""

    def __init__(self, need):
        self.need, self.seen, self.inside, self.most = need, [], 0, 0

    def pq1_paged_attention_workspace_bytes(self, *sizes):
        return self.need

    def pq1_paged_attention(self, *args):
        address, size, stream = args[-3:]
        if self.need and not address:
            return 1
        if size < self.need:
            return 8
        self.inside += 1
        self.most = max(self.most, self.inside)
        time.sleep(0.002)
        self.inside -= 1
        self.seen.append((address, size, stream))
        return 0


@pytest.fixture
def binding(monkeypatch):
    monkeypatch.setattr(pq1, "_raw_stream", lambda index: 77)
    monkeypatch.setattr(pq1, "_capturing", lambda: False)
    monkeypatch.setattr(pq1, "_attn_ws", {})
    args = (None, None, types.SimpleNamespace(dim=64), None, 1, None, None, 1, 1, 2, 1, 9, 1.0, 1, 0)
    return lambda lib: pq1._attend(lib, torch.device("cpu"), 2, args)


def test_workspace_of_a_stream_is_kept_and_grown(binding):
    lib = Recorder(2 << 20)
    binding(lib)
    binding(lib)
    assert lib.seen[0] == lib.seen[1] and lib.seen[0][1] == 2 << 20
    lib.need = 3 << 20
    binding(lib)
    assert lib.seen[2][1] == 3 << 20 and len(pq1._attn_ws) == 1


def test_captured_calls_take_no_workspace_of_a_stream(binding, monkeypatch):
    """Two captured calls, and eager ones of the same stream, share nothing that
    outlives the capture."""
    lib = Recorder(2 << 20)
    binding(lib)
    held = dict(pq1._attn_ws)
    monkeypatch.setattr(pq1, "_capturing", lambda: True)
    made = []
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(empty(*a, **k)) or made[-1])
    binding(lib)
    binding(lib)
    assert pq1._attn_ws == held
    assert len({a for a, _, _ in lib.seen}) == 3 and len(made) == 2
    lib.need = 0
    binding(lib)
    assert lib.seen[-1][:2] == (None, 0) and pq1._attn_ws == held


def test_calls_of_two_threads_on_one_stream_follow_one_another(binding):
    """The library enqueues parts and their join in one call, on one workspace:
    no other thread's call on it may come between."""
    lib = Recorder(2 << 20)
    threads = [threading.Thread(target=lambda: [binding(lib) for _ in range(10)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(lib.seen) == 40 and lib.most == 1
    assert len({a for a, _, _ in lib.seen}) == 1


@pytest.mark.parametrize("cls,name", [(pq1.KVCache, "k"), (pq1.KVCache, "v"), (pq1.Rope, "freqs")])
def test_tensors_whose_address_is_kept_cannot_be_exchanged(cls, name):
    """The calls would go on with the old tensor's memory."""
    held = object.__new__(cls)
    with pytest.raises(AttributeError):
        setattr(held, name, torch.zeros(4))
