"""An attention layer on 1-bit projections: a prompt in chunks, then tokens one
at a time, over a paged cache.

    python examples/attention_layer.py

A layer's step is four calls after the rotation of its input: the stacked
query/key/value projection, pq1_kv_append (queries and keys rotated by their
positions on the way), pq1_paged_attention, and the output projection with its
own rotation.  Chunks of a prompt use the bf16 GEMM, single tokens the fused
decode step; the attention calls are the same for both.  With norms=True queries
and keys are normed on the way into the cache, with bits=4 that holds 4-bit numbers
(pq1_kv4_append, pq1_kv4_attention), and with a window each token sees the last
`window` ones and the first `sinks`.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from gemm_hadamard_rotated_amd import pq1  # noqa: E402


class AttentionLayer:
    """Random 1-bit weights of the tested 27B model's head shapes."""

    def __init__(self, hidden=5120, heads=24, kv_heads=4, dim=256, rot=64, sections=(11, 11, 10),
                 pages=64, page_size=64, seed=0, device="cuda:0", norms=False, bits=16, window=0,
                 sinks=0):
        self.hidden, self.heads, self.kv_heads, self.dim = hidden, heads, kv_heads, dim
        self.window, self.sinks = window, sinks
        self.dev = torch.device(device)
        g = torch.Generator(device=self.dev).manual_seed(seed)
        self.qkv = self._weights((heads + 2 * kv_heads) * dim, hidden, g)
        self.out = self._weights(hidden, heads * dim, g)
        self.rope = pq1.Rope(rot, sections, freqs=pq1.rope_frequencies(rot, 1.0e6, self.dev),
                             interleaved=True)
        kind = pq1.KV4Cache if bits == 4 else pq1.KVCache
        self.cache = kind.empty(pages, page_size, kv_heads, dim, device=self.dev)
        self.append = pq1.pq1_kv4_append if bits == 4 else pq1.pq1_kv_append
        self.attend = pq1.pq1_kv4_attention if bits == 4 else pq1.pq1_paged_attention
        self.norm = None
        if norms:
            w = 1 + 0.1 * torch.randn(2, dim, device=self.dev, generator=g)
            self.norm = pq1.HeadNorm(w[0], w[1])

    def _weights(self, N, K, g):
        bits = torch.randint(-2 ** 31, 2 ** 31, (N, K // 32), device=self.dev, generator=g).to(
            torch.int32)
        scales = torch.rand(N, K // 128, device=self.dev, generator=g) * (1.5 / K ** 0.5)
        signs = torch.randint(0, 2, (K,), device=self.dev, generator=g).float() * 2 - 1
        return bits, scales, signs, pq1.pq1_pack_weights(bits, scales)

    @staticmethod
    def _project(x, weights):
        """x [T][K] fp32 -> [T][N] fp32."""
        bits, scales, signs, packed = weights
        if x.shape[0] == 1:
            return pq1.pq1_rotate_gemv_packed(x[0], signs, packed).unsqueeze(0)
        return pq1.pq1_gemm(pq1.pq1_rotate(x, signs, out_dtype=torch.bfloat16), bits, scales)

    def __call__(self, x, positions, slots, table, cu_q, kv_len, max_q, max_kv):
        """x [T][hidden] fp32, the new tokens of all sequences; returns the same shape."""
        H, Hk, D = self.heads, self.kv_heads, self.dim
        qkv = self._project(x, self.qkv)
        q, k, v = (qkv[:, a * D:b * D].unflatten(1, (b - a, D))
                   for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))
        q = self.append(self.cache, k, v, slots, positions=positions, rope=self.rope, q=q,
                        norm=self.norm)
        o = self.attend(q, self.cache, table, cu_q, kv_len, max_q, max_kv, window=self.window,
                        out_dtype=torch.float32, sinks=self.sinks)
        return self._project(o.view(x.shape[0], H * D), self.out)


class Sequence:
    """One sequence's pages and length, as a scheduler would keep them."""

    def __init__(self, layer, pages):
        self.page_size, self.dev = layer.cache.page_size, layer.dev
        self.pages = torch.tensor(pages, dtype=torch.int64, device=self.dev)
        self.table = self.pages.to(torch.int32).unsqueeze(0)
        self.length = 0

    def extend(self, n):
        """Arguments of the layer for the next n tokens."""
        at = torch.arange(self.length, self.length + n, device=self.dev)
        self.length += n
        slots = self.pages[at // self.page_size] * self.page_size + at % self.page_size
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=self.dev)
        return dict(positions=at.to(torch.int32).expand(3, n).contiguous(), slots=slots,
                    table=self.table, cu_q=i32([0, n]), kv_len=i32([self.length]), max_q=n,
                    max_kv=self.length)


def run(layer, x, pages, cuts):
    """x [T][hidden] through the layer, cut into chunks of these sizes."""
    seq, out, at = Sequence(layer, pages), [], 0
    for n in cuts:
        out.append(layer(x[at:at + n].contiguous(), **seq.extend(n)))
        at += n
    return torch.cat(out)


def main():
    layer = AttentionLayer()
    T = 1000
    g = torch.Generator(device=layer.dev).manual_seed(1)
    x = torch.randn(T, layer.hidden, device=layer.dev, generator=g)
    whole = run(layer, x, range(0, 16), [T])
    parts = run(layer, x, range(40, 24, -1), [512, 300, 180] + [1] * 8)
    torch.cuda.synchronize()
    size = whole.double().pow(2).mean().sqrt()
    error = (parts - whole).double().pow(2).mean().sqrt() / size
    print(f"chunks and single tokens against the whole prompt: {float(error):.2e} of its size")
    seq = Sequence(layer, range(0, 16))
    for label, n, times in (("chunk of 512 tokens", 512, 1), ("one token", 1, 100)):
        args = [seq.extend(n) for _ in range(times)]
        torch.cuda.synchronize()
        t = time.perf_counter()
        for a in args:
            layer(x[:n].contiguous(), **a)
        torch.cuda.synchronize()
        print(f"{label}: {(time.perf_counter() - t) / times * 1e6:.0f} us a layer")
    layer = AttentionLayer(norms=True, bits=4, window=256, sinks=4)
    run(layer, x, range(0, 16), [T])
    parts = run(layer, x, range(40, 24, -1), [512, 300, 180] + [1] * 8)
    print(f"normed, 4-bit cache, window of 256 and 4 first tokens: {list(parts.shape)}, "
          f"finite {bool(torch.isfinite(parts).all())}")
    return float(error)


if __name__ == "__main__":
    main()
