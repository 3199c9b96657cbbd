"""The expert-layer example: served, against the same layer in float32 on the
weights' values; trained, its gradients against autograd of the plain sums; and
the served layer captured in a graph."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import block_scaled_precision_02_amd as q  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dense(w):
    s = w.scales.repeat_interleave(128, 1).repeat_interleave(128, 2)
    return w.codes.float() * s


def rows(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * scales.repeat_interleave(128, 1)


def norm(x, g, eps):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * g.float()


def plain(layer, residual, ids, weights):
    """(the block's output, the new residual, the next block's A) in float32."""
    h = residual.float()
    x, out = norm(h, layer.before, layer.eps), torch.zeros_like(h)
    gu, down = dense(layer.gate_up), dense(layer.down)
    for t in range(h.shape[0]):
        for j, e in enumerate(ids[t].tolist()):
            if 0 <= e < layer.experts:
                g, u = (gu[e] @ x[t]).chunk(2)
                out[t] += weights[t, j] * (down[e] @ (torch.nn.functional.silu(g) * u))
    new = h + layer.alpha * layer.gate.float() * norm(out, layer.after, layer.eps)
    return out, new, norm(new, layer.following, layer.eps)


@pytest.mark.parametrize("tokens,experts,k", [(1, 16, 4), (7, 32, 8), (65, 8, 2), (300, 16, 4)])
def test_served(tokens, experts, k):
    import expert_layer as ex
    layer = ex.ExpertLayer(hidden=512, ffn=256, experts=experts, top_k=k, alpha=0.5, seed=tokens)
    r = torch.randn(tokens, 512, device="cuda").bfloat16()
    ids, weights = layer.route(r)
    want, new, z = plain(layer, r, ids, weights)
    codes, scales, _ = q.qgemm_rmsnorm_quant_f8_block(r, layer.before, layer.eps)
    x = layer.block(codes, scales, ids, weights)
    # e4m3 activations (steps of 2^-4 relative, errors of about 2.6% a value) go
    # through the first product and the second; the norm of the sum of two such
    # independent errors is under 4%, and each factor of silu(g) u carries the first
    assert float((x.float() - want).norm() / want.norm()) < 0.08
    own = r.clone()
    codes, scales = layer(own)
    # the residual keeps its part exactly, the block's normed output is half of it or less
    assert float((own.float() - new).norm() / new.norm()) < 0.05
    # and one more quantisation of the whole
    assert float((rows(codes, scales) - z).norm() / z.norm()) < 0.08


def test_one_rank_of_two():
    """Each rank's experts give their share of the sum."""
    import expert_layer as ex
    layer = ex.ExpertLayer(hidden=512, ffn=256, experts=16, top_k=4, seed=5)
    r = torch.randn(40, 512, device="cuda").bfloat16()
    ids, weights = layer.route(r)
    codes, scales, _ = q.qgemm_rmsnorm_quant_f8_block(r, layer.before, layer.eps)
    whole = layer.block(codes, scales, ids, weights).float()
    parts = []
    for first in (0, 8):
        half = ex.ExpertLayer(hidden=512, ffn=256, experts=16, top_k=4, seed=5)
        half.experts = 8
        for w in (half.gate_up, half.down):
            w.codes, w.scales = w.codes[first:first + 8].contiguous(), w.scales[first:first + 8].contiguous()
        parts.append(half.block(codes, scales, (ids - first).int(), weights).float())
    # the same rows; two roundings of bf16 and the order of the sum
    size = parts[0].abs() + parts[1].abs()
    assert bool(((parts[0] + parts[1] - whole).abs() <= 2.0 ** -7 * size + 1e-6).all())


def test_captured():
    import expert_layer as ex
    layer = ex.ExpertLayer(hidden=512, ffn=256, experts=16, top_k=4, seed=2)
    r = torch.randn(33, 512, device="cuda").bfloat16()
    ids, weights = layer.route(r)
    codes, scales, _ = q.qgemm_rmsnorm_quant_f8_block(r, layer.before, layer.eps)
    layer.block(codes, scales, ids, weights)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.block(codes, scales, ids, weights)
    for seed in range(3):
        # other choices, so other counts, under the same graph
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        ids.copy_(torch.rand(33, 16, device="cuda", generator=g).argsort(1)[:, :4] - seed)
        want = layer.block(codes, scales, ids, weights)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_gradients():
    import expert_layer as ex
    T, k, E, H = 24, 3, 6, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ids = torch.rand(T, E, device="cuda", generator=g).argsort(1)[:, :k].int() - 1      # one of them not here
    offsets, order, position = q.qgemm_moe_sort(ids, E - 1)
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16().requires_grad_()
    w = torch.rand(T, k, device="cuda", generator=g).requires_grad_()
    scale = torch.randn(E - 1, H, device="cuda", generator=g).bfloat16().requires_grad_()   # an expert: a scale for each channel
    dout = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    live = int(offsets[-1])
    xs = ex.gather(x, position)[:live]
    of = torch.repeat_interleave(torch.arange(E - 1, device="cuda"), (offsets[1:] - offsets[:-1]).long())
    y = torch.cat([xs * scale[of], torch.zeros(T * k - live, H, device="cuda").bfloat16()])
    out = ex.combine(y, position, w)
    out.backward(dout)
    # the same in 64 bits, token by token
    X, W, S = (t.detach().double().requires_grad_() for t in (x, w, scale))
    rows_ = []
    for t in range(T):
        acc = torch.zeros(H, dtype=torch.float64, device="cuda")
        for j, e in enumerate(ids[t].tolist()):
            if 0 <= e < E - 1:
                acc = acc + W[t, j] * (X[t] * S[e])
        rows_.append(acc)
    want = torch.stack(rows_)
    want.backward(dout.double())
    # Each value passes at most four roundings to bf16 (the row, its gradient, the
    # product with the expert's scale, the sum), relative to the terms' sizes
    tol = 5 * 2.0 ** -8

    terms = torch.stack([sum(((W[t, j] * X[t] * S[e]).abs() for j, e in enumerate(ids[t].tolist()) if 0 <= e < E - 1),
                             torch.zeros(H, dtype=torch.float64, device="cuda")) for t in range(T)])
    assert bool(((out.double() - want).abs() <= tol * terms + 1e-12).all())
    for a, b in ((x.grad, X.grad), (w.grad, W.grad), (scale.grad, S.grad)):
        assert float((a.double() - b).norm() / b.norm()) < tol
    gone = position < 0
    assert bool(gone.any()) and not bool(w.grad[gone].any())
