"""Keys of a 4-bit cache turned by angles of any size."""
import pytest
import torch

import attention_reference as ref
import kv4_reference as ref4
from test_gpu_kv4 import BF16, F32, pq, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairing", ["halves", "adjacent"])
def test_keys_turned_by_any_angle_keep_their_length(pq, dev, pairing):  # noqa: F811
    """Far out an angle's own rounding is more than a turn: any turn will do, but it has
    to be one.  Pairs (1, 1) stay of length sqrt(2): the larger of two such numbers lies in
    [1, sqrt(2)], so every scale is 2^-2, whose codes up to 1.5 are off by 0.25 at most."""
    D, page = 64, 8
    freqs = 10.0 ** torch.linspace(-3, 30, D // 2, dtype=torch.float64)
    pos = torch.tensor([0, 1, -1, 77, 2 ** 20 + 1, 2 ** 31 - 1, -2 ** 31, -12345], dtype=torch.int32)
    T = pos.numel()
    cache = pq.KV4Cache.empty(2, page, 1, D, BF16, dev)
    x = torch.ones(T, 1, D)
    at = torch.arange(T)
    rope = pq.Rope(D, freqs=freqs.to(dev), pairing=pairing)
    q = pq.pq1_kv4_append(cache, x.to(dev), x.to(dev), at.to(dev), positions=pos.to(dev), rope=rope,
                          q=x.to(dev))
    assert bool((rows(cache.k_scale, at, page) == 125).all())
    k = ref4.values(rows(cache.k, at, page), rows(cache.k_scale, at, page))
    lo = k[..., :D // 2] if pairing == "halves" else k[..., 0::2]
    hi = k[..., D // 2:] if pairing == "halves" else k[..., 1::2]
    assert float((torch.hypot(lo, hi) - 2.0 ** 0.5).abs().max()) <= 0.25 * 2.0 ** 0.5
    # the queries' pairs: rounded to bf16, 2^-8 of each number besides 2^-20
    y = q.double().cpu()
    lo = y[..., :D // 2] if pairing == "halves" else y[..., 0::2]
    hi = y[..., D // 2:] if pairing == "halves" else y[..., 1::2]
    assert float((torch.hypot(lo, hi) - 2.0 ** 0.5).abs().max()) <= 2.0 ** 0.5 * (2.0 ** -8 + 2.0 ** -19)


def test_keys_turned_by_large_angles(pq, dev):  # noqa: F811
    """Angles up to 2^47 radians: the codes of the formula's values.  Values are off by a
    few 2^-53 of the pair; none of the drawn ones is within 2^-40 of a border."""
    D, page, T = 64, 8, 64
    g = torch.Generator().manual_seed(4)
    freqs = 2.0 ** torch.linspace(-20, 16, D // 2, dtype=torch.float64)
    pos = torch.randint(-2 ** 31, 2 ** 31, (T,), generator=g).to(torch.int32)
    x = torch.randn(T, 1, D, generator=g)
    y, _ = ref.rotate(x, pos, freqs, (D // 2,), "halves", False)
    want, byte = ref4.quantise(y, BF16)
    for nudge in (1 - 2.0 ** -40, 1 + 2.0 ** -40):
        assert torch.equal(ref4.quantise(y * nudge, BF16)[0], want), "a value next to a border"
    cache = pq.KV4Cache.empty(T // page, page, 1, D, BF16, dev)
    at = torch.arange(T)
    pq.pq1_kv4_append(cache, x.to(dev), x.to(dev), at.to(dev), positions=pos.to(dev),
                      rope=pq.Rope(D, freqs=freqs.to(dev)))
    assert torch.equal(rows(cache.k_scale, at, page), byte)
    got = ref4.values(rows(cache.k, at, page), rows(cache.k_scale, at, page))
    assert torch.equal(got, want)
