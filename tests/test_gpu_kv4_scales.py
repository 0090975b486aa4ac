"""Attention over 4-bit caches whose scale bytes are any of the 256, on the GPU: what a
64-bit form gives over the values that reading the cache back gives."""
import pytest
import torch

import attention_reference as ref
import kv4_reference as ref4
from test_gpu_attention import BF16, F16, F32, STATED, check, pq  # noqa: F401
from test_gpu_attention_windows import Pages4

pytestmark = pytest.mark.gpu

# Past the append's range some codes stand for no finite number of the type: from 4, 2, 1
# and 0.5 on in f16 (2^16 is none), from 4 and 2 on in bf16 (2^128 is none).
BYTES = {F16: (0, 90, 141, 142, 143, 144, 150, 255), BF16: (0, 20, 253, 254, 255)}
LEAST_ODD = {F16: {141: 6, 142: 4, 143: 2, 144: 1, 150: 1}, BF16: {253: 6, 254: 4}}


def put(s, which, key, byte, finite, seed):
    """One row of sequence 0, all heads: groups of this byte in turn with codes of finite
    values alone and, unless `finite`, any codes; s.k or s.v become what that is."""
    g = torch.Generator().manual_seed(seed)
    shape = (s.Hk, s.D // 32, 32)
    code = torch.randint(0, 8, shape, generator=g)
    limit = LEAST_ODD[s.dtype].get(byte, 8)
    low = code % limit
    code = low if finite else torch.where((torch.arange(s.D // 32) % 2 == 0)[:, None], low, code)
    code = (code + 8 * torch.randint(0, 2, shape, generator=g)).flatten(1).to(torch.uint8)
    codes = code[:, 0::2] + 16 * code[:, 1::2]
    scales = torch.full((s.Hk, s.D // 32), byte, dtype=torch.uint8)
    p, r = int(s.table[0, key // s.page]), key % s.page
    held = (s.cache.k, s.cache.k_scale) if which == "k" else (s.cache.v, s.cache.v_scale)
    held[0][p, :, r] = codes.to(s.dev)
    held[1][p, :, r] = scales.to(s.dev)
    (s.k if which == "k" else s.v)[0][key] = ref4.values(codes, scales).to(s.dtype)


def slots_of(s):
    """Of all keys of sequence 0."""
    j = torch.arange(s.kvs[0])
    return s.table[0, j // s.page].long() * s.page + j % s.page


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("rows,D,page", [(1, 64, 16), (4, 128, 4), (30, 256, 32), (120, 128, 32),
                                         (70, 64, 8), (40, 256, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 5)])
def test_values_under_any_scale(pq, dev, rows, D, page, dt, window, sinks):  # noqa: F811
    """Rows that all, some or one row sees: finite values count, infinities and NaN reach
    the rows that see them and no others."""
    kv = rows + 90
    for byte in BYTES[dt]:
        for finite in (True, False):
            if finite and byte == 255:
                continue
            s = Pages4(pq, dev, [rows, 3], [kv, 33], 1, 2, D, page, dt, seed=5)
            for n, key in enumerate((2, kv - rows, kv - 1 - rows // 2, kv - 1)):
                put(s, "v", key, byte, finite, 100 * byte + n)
            k, v = pq.pq1_kv4_read(s.cache, slots_of(s).to(dev))
            assert torch.equal(v.cpu().nan_to_num(9), s.v[0].nan_to_num(9)), f"byte {byte}: read"
            for stated in STATED:
                for out in (dt, F32):
                    got = s.run(max_kv=stated, window=window, sinks=sinks, out_dtype=out)
                    s.check(got, True, window, sinks,
                            where=f"byte {byte}, finite {finite}, stated {stated}, {out}")


@pytest.mark.parametrize("dt", [BF16, F16], ids=["bf16", "f16"])
@pytest.mark.parametrize("rows,D,page", [(1, 64, 16), (4, 128, 4), (30, 256, 32), (120, 128, 32)])
def test_keys_under_any_scale(pq, dev, rows, D, page, dt):  # noqa: F811
    """Keys likewise: queries so small that scores of finite keys are ordinary numbers."""
    kv = rows + 90
    for byte in BYTES[dt]:
        s = Pages4(pq, dev, [rows, 3], [kv, 33], 1, 2, D, page, dt, seed=6)
        for n, key in enumerate((2, kv - rows, kv - 1)):
            put(s, "k", key, byte, True, 100 * byte + n)
        least = min(byte - 127, 120 if dt == BF16 else 13)
        if least > 0:
            s.q = (s.q.double().sign() * 2.0 ** -least).to(dt)
        e, w, spread = ref4.attention(s.q[:rows], s.k[0], s.v[0], D ** -0.5, True, 0, 0)
        vmax = float(s.v[0].double().abs().max())
        for stated in STATED:
            for out in (dt, F32):
                got = s.run(max_kv=stated, out_dtype=out)
                # One key takes nearly all of a row here.  bf16 probabilities are carried times
                # 2^-20, with the row's largest at 2^-20 or more: what is below 2^-126 may become
                # zero, and of three parts two may be kept 2^-126 too large.  So each probability
                # is off by at most 2^-124 / 2^-20 of the row's largest besides.
                b = ref.attention_bound(e, w, spread, kv, vmax, D, dt, out)
                if dt == BF16:
                    b = b + kv * 2.0 ** -104 * vmax
                check(got[:rows], e, b, f"byte {byte}, stated {stated}, {out}")


def test_a_page_that_is_none_beside_large_scales(pq, dev):  # noqa: F811
    """A tile with a page outside the cache: rows that see it are NaN, the others keep
    the finite values under scales past the append's range."""
    rows, D, page = 60, 128, 16
    kv = 128
    for stated in STATED:
        s = Pages4(pq, dev, [rows], [kv], 1, 2, D, page, F16, seed=8)
        for n, key in enumerate((70, 75, 111)):
            put(s, "v", key, 141, True, n)
        want = s.run(max_kv=stated)
        s.check(want, where=f"stated {stated}")
        s.table[0, kv // page - 1] = s.pages          # the last 16 keys
        got = s.run(max_kv=stated)
        sees = torch.arange(rows) + kv - rows >= kv - page
        assert bool(torch.isnan(got.cpu()[sees]).all())
        assert torch.equal(got.cpu()[~sees], want.cpu()[~sees])
