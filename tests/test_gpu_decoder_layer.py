"""The decoder-layer example against the same layer in float32: a ragged prompt
and then single tokens, with the cache carried along."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _dense(linear):
    """The weight's values, float32 [n, k]."""
    t = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")
    n = linear.codes.shape[0]
    w = torch.stack((linear.codes & 15, linear.codes >> 4), 2).view(n, -1)
    return (t[w.int()].view(n, -1, 32) * torch.exp2(linear.scales.float() - 127)[..., None]).view(n, -1)


class Plain:
    """The layer in float32, the keys and values kept as they are."""

    def __init__(self, layer, batch):
        self.l, self.k, self.v = layer, [[] for _ in range(batch)], [[] for _ in range(batch)]

    def _norm(self, h, g):
        return h * torch.rsqrt(h.square().mean(1, keepdim=True) + self.l.eps) * g.float()

    def __call__(self, x, residual, counts):
        l, d = self.l, self.l.head_dim
        h = x.float() + residual.float()
        qkv = self._norm(h, l.norm1) @ _dense(l.qkv).t()
        nq, nk, at, outs = l.heads * d, l.kv_heads * d, 0, []
        for b, n in enumerate(counts):
            rows = qkv[at:at + n]
            at += n
            self.k[b].append(rows[:, nq:nq + nk].view(n, -1, d))
            self.v[b].append(rows[:, nq + nk:].view(n, -1, d))
            k, v = (torch.cat(t).repeat_interleave(l.heads // l.kv_heads, 1) for t in (self.k[b], self.v[b]))
            s = torch.matmul(rows[:, :nq].view(n, -1, d).transpose(0, 1), k.permute(1, 2, 0).contiguous()) * d ** -0.5
            total = k.shape[0]
            hide = torch.arange(total, device="cuda")[None] > torch.arange(total - n, total, device="cuda")[:, None]
            p = torch.softmax(s.masked_fill(hide, float("-inf")), 2)
            outs.append(torch.matmul(p, v.transpose(0, 1).contiguous()).transpose(0, 1).reshape(n, nq))
        h = h + torch.cat(outs) @ _dense(l.out).t()
        gu = self._norm(h, l.norm2) @ _dense(l.gate_up).t()
        return (torch.nn.functional.silu(gu[:, :l.ffn]) * gu[:, l.ffn:]) @ _dense(l.down).t(), h


@pytest.mark.parametrize("fmt", [0, 1])
def test_prompt_then_tokens(fmt):
    import decoder_layer as ex
    layer = ex.DecoderLayer(hidden=512, ffn=1024, heads=8, kv_heads=2, head_dim=64, seed=3)
    cache = layer.cache(24, 16, fmt)
    table = torch.randperm(24, device="cuda").int().view(3, 8)
    plain, lens = Plain(layer, 3), [0, 0, 0]
    for step, counts in enumerate(([70, 33, 1], [1, 1, 1], [1, 1, 1], [5, 1, 30])):
        g = torch.Generator(device="cuda")
        g.manual_seed(step)
        lens = [a + b for a, b in zip(lens, counts)]
        x = torch.randn(sum(counts), 512, device="cuda", generator=g).bfloat16()
        r = torch.randn(sum(counts), 512, device="cuda", generator=g).bfloat16()
        want, h = plain(x, r, counts)
        y = layer(x, r, cache, table, ex.offsets(counts), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                  max(counts), max(lens))
        # e4m3 activations (relative steps of 2^-4, errors of about 2.6% a value)
        # go through three products, the cache adds 8-bit keys and values: the
        # layer's output within 10% of the float32 one, the residual, which holds
        # x exactly and one product of the attention, within 5%
        assert float((y.float() - want).norm() / want.norm()) < 0.10, step
        assert float((r.float() - h).norm() / h.norm()) < 0.05, step
