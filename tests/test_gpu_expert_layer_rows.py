"""GPU test of the expert-layer example's way there and back on one rank of
several: experts applied to every row that the gather has room for, the rows
without a choice among them, whatever new memory holds."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import block_scaled_precision_02_amd as q  # noqa: E402


@pytest.fixture(autouse=True)
def _new_memory_is_nan():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert torch.utils.deterministic.fill_uninitialized_memory
    torch.use_deterministic_algorithms(True)
    yield
    torch.use_deterministic_algorithms(False)


def test_rows_without_a_choice():
    import expert_layer as ex
    T, k, E, H = 24, 3, 6, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    ids = torch.rand(T, E, device="cuda", generator=g).argsort(1)[:, :k].int() - 3       # half of them not here
    offsets, order, position = q.qgemm_moe_sort(ids, E - 3)
    live = int(offsets[-1])
    assert 0 < live < T * k and bool(torch.empty(8, device="cuda").isnan().all())
    x = torch.randn(T, H, device="cuda", generator=g).bfloat16().requires_grad_()
    w = torch.rand(T, k, device="cuda", generator=g).requires_grad_()
    scale = torch.randn(H, device="cuda", generator=g).requires_grad_()                  # one for all experts
    xs = ex.gather(x, position)
    assert not bool(xs[live:].any()) and bool(xs[:live].isfinite().all())
    out = ex.combine((xs * scale).bfloat16(), position, w)
    dout = torch.randn(T, H, device="cuda", generator=g).bfloat16()
    out.backward(dout)
    X, W, S = (t.detach().double().requires_grad_() for t in (x, w, scale))
    here = (position >= 0).double()
    ((W * here).sum(1)[:, None] * X * S).backward(dout.double())
    # bf16 roundings of the rows, their gradients and the result: as many as values
    # pass, 2^-8 of each term
    for a, b in ((x.grad, X.grad), (w.grad, W.grad), (scale.grad, S.grad)):
        assert bool(a.isfinite().all())
        assert float((a.double() - b).norm() / b.norm()) < 5 * 2.0 ** -8
