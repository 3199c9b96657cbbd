"""A layer of experts served in FP8 blockscale, and its way to the experts and
back in training.

    python examples/expert_layer.py [--tokens 64] [--experts 64] [--top-k 8]

Served (ExpertLayer), the block between two norms:

    A            from the norm before the block (here qgemm_rmsnorm_quant_f8_block)
    ids, w       top-k of the router's logits         torch
    order        the choices by expert                qgemm_moe_sort
    g, u         = A[tokens of the rows] . Wgu[e]     qgemm_f8_blockscale_grouped, rows through the order
    B            = silu(g) u, quantised               qgemm_swiglu_quant_f8_block
    y            = B . Wdown[e]                       qgemm_f8_blockscale_grouped
    x            = sum of a token's rows by w         qgemm_moe_combine
    h, A'        = r + alpha gate norm(x), and the norm before the next block, quantised
                                                      qgemm_postnorm_quant_f8_block

Trained (gather, combine): the same way there and back as autograd functions
around experts of the program's own.  Random weights and inputs.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_02_amd as q  # noqa: E402


class Experts:
    """FP8 blockscale weights of every expert, [experts, n, k]: e4m3 codes with
    one fp32 scale for each 128 x 128 block."""

    def __init__(self, w):
        e, n, k = w.shape
        b = w.float().view(e, n // 128, 128, k // 128, 128)
        self.scales = (b.abs().amax((2, 4)) / 448.0).contiguous()
        self.codes = (b / self.scales[:, :, None, :, None]).view(e, n, k).to(torch.float8_e4m3fn)

    def __call__(self, codes, scales, offsets, **kw):
        return q.qgemm_f8_blockscale_grouped(codes, self.codes, scales, self.scales, offsets, **kw)


class ExpertLayer:
    def __init__(self, hidden=2048, ffn=1024, experts=64, top_k=8, alpha=1.0, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def randn(*s):
            return torch.randn(*s, device="cuda", generator=gen)
        self.hidden, self.ffn, self.experts, self.top_k, self.alpha, self.eps = hidden, ffn, experts, top_k, alpha, 1e-6
        self.router = (randn(experts, hidden) * hidden ** -0.5).bfloat16()
        self.gate_up = Experts(randn(experts, 2 * ffn, hidden) * hidden ** -0.5)
        self.down = Experts(randn(experts, hidden, ffn) * ffn ** -0.5)
        self.before, self.after, self.following = ((1 + 0.1 * randn(hidden)).bfloat16() for _ in range(3))
        self.gate = torch.tanh(1 + 0.1 * randn(hidden)).bfloat16()

    def route(self, h):
        """ids int32 and weights fp32 [tokens, top_k] of the normed residual."""
        x = h.float() * torch.rsqrt(h.float().square().mean(1, keepdim=True) + self.eps) * self.before.float()
        top, ids = (x @ self.router.float().t()).topk(self.top_k, dim=1)
        return ids.int(), torch.softmax(top, 1)

    def block(self, codes, scales, ids, weights):
        """The experts' share: quantised rows of the tokens -> bf16 [tokens, hidden]."""
        offsets, order, position = q.qgemm_moe_sort(ids, self.experts)
        gu = self.gate_up(codes, scales, offsets, order=order)
        codes, scales = q.qgemm_swiglu_quant_f8_block(gu, count=offsets[-1:])
        return q.qgemm_moe_combine(self.down(codes, scales, offsets), position, weights)

    def __call__(self, residual):
        """residual bf16 [tokens, hidden], updated in place.  Returns the next
        block's A operand and its scales."""
        codes, scales, _ = q.qgemm_rmsnorm_quant_f8_block(residual, self.before, self.eps)
        x = self.block(codes, scales, *self.route(residual))
        codes, scales, _ = q.qgemm_postnorm_quant_f8_block(x, residual, self.after, self.following, self.eps,
                                                           gate=self.gate, alpha=self.alpha, residual_out=residual)
        return codes, scales


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, position):
        ctx.save_for_backward(position)
        # rows without a choice are zeros: what they hold meets a zero gradient in
        # the experts' weights' gradients
        xs = torch.zeros(position.numel(), x.shape[1], dtype=x.dtype, device=x.device)
        return q.qgemm_moe_gather(x, position, out=xs)

    @staticmethod
    def backward(ctx, dxs):
        return q.qgemm_moe_combine(dxs.contiguous(), *ctx.saved_tensors), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, position, weights):
        ctx.save_for_backward(y, position, weights)
        return q.qgemm_moe_combine(y, position, weights)

    @staticmethod
    def backward(ctx, dout):
        y, position, weights = ctx.saved_tensors
        dy, dweights = q.qgemm_moe_combine_grad(dout.contiguous(), y, position, weights, dY=torch.zeros_like(y))
        return dy, None, dweights


def gather(x, position):
    """The tokens' rows in order of experts, bf16 [tokens * top_k, hidden]; zeros
    behind the last one."""
    return _Gather.apply(x, position)


def combine(y, position, weights):
    """The experts' rows summed back with weights, bf16 [tokens, hidden]."""
    return _Combine.apply(y, position, weights)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--top-k", type=int, default=8)
    a = ap.parse_args()
    layer = ExpertLayer(experts=a.experts, top_k=a.top_k)
    r = torch.randn(a.tokens, layer.hidden, device="cuda").bfloat16()
    layer(r)                                                # once untimed
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(20):
        codes, scales = layer(r)
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / 20
    assert bool(scales.isfinite().all())
    print(f"{a.tokens} tokens, {a.top_k} of {a.experts} experts: {t * 1e6:.0f} us a layer, {a.tokens / t:.0f} tokens/s")


if __name__ == "__main__":
    main()
