"""The attention-layer calls on the GPU at the edges of what they allow: hints
of any size, chunks and caches beyond the hints, values and probabilities at the
ends of their types' ranges, workspaces in graphs."""
import pytest
import torch

import attention_reference as ref
from test_gpu_attention import BF16, F16, F32, Batch, check, pq  # noqa: F401  (pq: fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stated", [0x7fff0000, 0x7fffff01, 2 ** 31 - 1, 2 ** 62])
@pytest.mark.parametrize("B,rows,G", [(64, 1, 6), (1, 150, 8), (2, 1, 2)])
def test_longest_cache_stated_without_limit(pq, dev, B, rows, G, stated):
    """A caller that knows no limit states the largest number."""
    Hk = 4 if B > 1 else 32
    s = Batch(pq, dev, [rows] * B, [9 + 3 * (b % 5) for b in range(B)], Hk, G, 64, 16, BF16)
    s.check(s.run(max_kv=stated), where=f"stated {stated}")
