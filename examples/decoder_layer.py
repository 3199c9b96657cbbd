"""One decoder layer served in low precision: prompts, then single tokens.

    python examples/decoder_layer.py [--batch 8] [--prompt 512] [--tokens 32]

Weights are MXFP4 (e2m1 with a ue8m0 scale per 32), the cache is 8-bit, the
activations of the wide projections MXFP8:

    h, A   = rms norm of x + residual, as MXFP8        qgemm_rmsnorm_quant_mx
    q k v  = A . Wqkv                                  qgemm_mx_mixed
    cache += k, v                                      qgemm_kv8_append
    o      = attention(q, cache)                       qgemm_kv8_attention
    x      = o . Wo        bf16 x 4-bit weights        qgemm_w4_matvec_mx (up to 64 rows)
                           more rows: MXFP8            qgemm_quant_mx, qgemm_mx_mixed
    h, A   = rms norm of x + h, as MXFP8
    g, u   = A . Wgu;  x = (silu(g) u) . Wdown         as above

Random weights and inputs.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_02_amd as q  # noqa: E402

E4M3, E2M1 = q.QGEMM_MX_E4M3, q.QGEMM_MX_E2M1
# The matvec's most; it is the faster one here up to that (2048 x 7168, 64 rows:
# 31 us against 44 for the quantiser and the GEMM; 17 rows: 14 against 40).
MATVEC_ROWS = 64


class Linear:
    """An MXFP4 weight [n, k]."""

    def __init__(self, w):
        self.codes, self.scales = q.qgemm_quant_mx(E2M1, w.bfloat16())

    def wide(self, codes, scales):
        """MXFP8 rows through the GEMM."""
        return q.qgemm_mx_mixed(E4M3, E2M1, codes, self.codes, scales, self.scales, q.QGEMM_MX_BSCALE_1x32)

    def __call__(self, x):
        """bf16 rows: the matvec for a decode step's, else quantised for the GEMM."""
        if x.shape[0] <= MATVEC_ROWS:
            return q.qgemm_w4_matvec_mx(x, self.codes, self.scales, q.QGEMM_MX_BSCALE_1x32)
        return self.wide(*q.qgemm_quant_mx(E4M3, x))


class DecoderLayer:
    def __init__(self, hidden=2048, ffn=7168, heads=16, kv_heads=2, head_dim=128, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def weight(n, k):
            return Linear(torch.randn(n, k, device="cuda", generator=gen) * k ** -0.5)
        self.heads, self.kv_heads, self.head_dim, self.ffn, self.eps = heads, kv_heads, head_dim, ffn, 1e-6
        self.qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, heads * head_dim)
        self.gate_up = weight(2 * ffn, hidden)
        self.down = weight(hidden, ffn)
        self.norm1, self.norm2 = ((1 + 0.1 * torch.randn(hidden, device="cuda", generator=gen)).bfloat16()
                                  for _ in range(2))

    def cache(self, blocks, block=64, fmt=q.QGEMM_KV8_E4M3):
        return q.KV8Cache.empty(blocks, self.kv_heads, self.head_dim, block, fmt)

    def __call__(self, x, residual, cache, table, cu, lens, max_q, max_kv):
        """x, residual bf16 [tokens, hidden]: the layer before's output and the
        residual stream (updated in place).  Returns this layer's output."""
        tokens, d = x.shape[0], self.head_dim
        codes, scales, _ = q.qgemm_rmsnorm_quant_mx(E4M3, x, self.norm1, self.eps, residual=residual,
                                                    residual_out=residual)
        qkv = self.qkv.wide(codes, scales)
        nq, nk = self.heads * d, self.kv_heads * d
        k, v = qkv[:, nq:nq + nk].view(tokens, -1, d), qkv[:, nq + nk:].view(tokens, -1, d)
        q.qgemm_kv8_append(cache, k, v, table, cu, lens, max_q)
        o = q.qgemm_kv8_attention(cache, qkv[:, :nq].view(tokens, -1, d), table, cu, lens, max_q, max_kv)
        x = self.out(o.view(tokens, nq))
        codes, scales, _ = q.qgemm_rmsnorm_quant_mx(E4M3, x, self.norm2, self.eps, residual=residual,
                                                    residual_out=residual)
        gu = self.gate_up.wide(codes, scales)
        return self.down(torch.nn.functional.silu(gu[:, :self.ffn]) * gu[:, self.ffn:])


def offsets(counts):
    """int32 [batch + 1] on the GPU: where each sequence's new tokens start."""
    return torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0).int().cuda()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=32)
    a = ap.parse_args()
    layer = DecoderLayer()
    hidden, block = 2048, 64
    width = -(-(a.prompt + a.tokens) // block)
    cache = layer.cache(a.batch * width, block)
    table = torch.arange(a.batch * width, dtype=torch.int32, device="cuda").view(a.batch, width)

    def step(count, length):
        x = torch.randn(a.batch * count, hidden, device="cuda").bfloat16()
        lens = torch.full((a.batch,), length, dtype=torch.int32, device="cuda")
        return layer(x, torch.randn_like(x), cache, table, offsets([count] * a.batch), lens, count, length)

    for name, count, steps, first in (("prompt", a.prompt, 1, a.prompt), ("decode", 1, a.tokens, a.prompt + 1)):
        step(count, first)                                  # once untimed; the same tokens are written again
        torch.cuda.synchronize()
        t = time.perf_counter()
        for i in range(steps):
            y = step(count, first + i)
        torch.cuda.synchronize()
        t = (time.perf_counter() - t) / steps
        assert bool(y.isfinite().all())
        print(f"{name}: {a.batch} x {count} tokens, {t * 1e6:.0f} us a layer, {a.batch * count / t:.0f} tokens/s")


if __name__ == "__main__":
    main()
