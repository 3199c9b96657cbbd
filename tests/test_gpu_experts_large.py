"""GPU tests of the operators of a layer of experts where one launch cannot hold
all threads, or holds as many pieces as its 32-bit index counts: rows at the
parts' ends against calls on those rows alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

from tests.test_gpu_postnorm import call as postnorm  # noqa: E402
from tests.test_gpu_swiglu import call as swiglu, parts_of  # noqa: E402

KINDS = ["i8", "f8", "block", "mx8", "mx4"]


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def bits(t):
    return t.contiguous().view(torch.uint8)


def test_exchange_of_many_tokens():
    T, H = (1 << 23) + 37, 8
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, y, r = (torch.randn(T, H, device="cuda", generator=g).bfloat16() for _ in range(3))
    w = torch.rand(T, 1, device="cuda", generator=g)
    position = torch.randperm(T, device="cuda", generator=g).int().view(T, 1)
    position[::5] = -1
    live, p = (position >= 0).view(-1), position.view(-1).clamp(min=0).long()
    zero = torch.zeros_like(x)
    xs = q.qgemm_moe_gather(x, position, out=torch.zeros_like(x))
    want = torch.zeros_like(x)
    want[p[live]] = x[live]
    assert torch.equal(xs, want)
    own = r.clone()
    got = q.qgemm_moe_combine(y, position, w, residual=own, out=own)
    want = torch.addcmul(r.double(), w.double(), torch.where(live[:, None], y[p], zero).double())
    # one binary32 rounding, one of bf16
    assert bool(((got.double() - want).abs() <= want.abs() * 2.0 ** -8 + (r.double().abs() + y[p].double().abs()) * 2.0 ** -23).all())
    dy, dw = q.qgemm_moe_combine_grad(r, y, position, w, dY=torch.zeros_like(y))
    want = torch.zeros_like(y)
    want[p[live]] = (w * r.float()).bfloat16()[live]
    assert torch.equal(dy, want)
    dot = torch.where(live, (r.double() * y[p].double()).sum(1), 0.0)
    size = (r.double() * y[p].double()).abs().sum(1)
    assert bool(((dw.view(-1).double() - dot).abs() <= H * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("kind", KINDS)
def test_swiglu_of_many_rows(kind):
    M, I = (1 << 24) + 5, 128 if kind == "block" else 32
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn(M, 2 * I, device="cuda", generator=g, dtype=torch.bfloat16)
    last = (1 << 24) + 3
    parts = parts_of(kind, I)
    out = torch.full((M, I // 2 if kind == "mx4" else I), 77, dtype=torch.int8 if kind == "i8" else torch.uint8,
                     device="cuda")
    scale = torch.full((M,) if kind in ("i8", "f8") else (M, parts), 9, device="cuda",
                       dtype=torch.uint8 if kind.startswith("mx") else torch.float32)
    swiglu(kind, x, count=torch.tensor([last], dtype=torch.int32, device="cuda"), out=out, scale=scale)
    for lo in (0, (1 << 23) - 3, (1 << 24) - 3):
        hi = min(lo + 6, last)
        for a, b in zip((out, scale), swiglu(kind, x[lo:hi].contiguous())):
            assert torch.equal(bits(a[lo:hi]), bits(b)), lo
    assert bool((out[last:] == 77).all()) and bool((scale[last:] == 9).all())


@pytest.mark.parametrize("kind", ["mx8", "mx4", "block"])
def test_swiglu_of_as_many_pieces_as_a_launch_counts(kind):
    """2^31 pieces of 8 in the first launch."""
    I = 16384
    per = (1 << 31) // (I // 8)
    M = per + 3
    x = torch.zeros(M, 2 * I, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    rows = [0, 1, per // 2 - 1, per // 2, per - 2, per - 1, per, M - 1]
    for r in rows:
        x[r] = torch.randn(2 * I, device="cuda", generator=g).bfloat16()
    codes, scale = swiglu(kind, x)
    want = swiglu(kind, x[rows])
    assert torch.equal(bits(codes[rows]), bits(want[0])) and torch.equal(bits(scale[rows]), bits(want[1]))
    rest = torch.ones(M, dtype=torch.bool, device="cuda")
    rest[rows] = False
    assert not bool(scale.float().sum(1)[rest].any())


@pytest.mark.parametrize("kind", KINDS)
def test_postnorm_of_many_rows(kind):
    M, K = (1 << 23) + 5, 128 if kind == "block" else 32
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    y, r = (torch.randn(M, K, device="cuda", generator=g, dtype=torch.bfloat16) for _ in range(2))
    gp, gm, gate = (torch.randn(K, device="cuda", generator=g).bfloat16() for _ in range(3))
    got = postnorm(kind, y, r, gp, gm, gate=gate, alpha=0.5)
    for lo in (0, (1 << 22) - 3, (1 << 23) - 3):
        hi = min(lo + 8, M)
        want = postnorm(kind, y[lo:hi].contiguous(), r[lo:hi].contiguous(), gp, gm, gate=gate, alpha=0.5)
        for a, b in zip(got, want):
            assert torch.equal(bits(a[lo:hi]), bits(b)), lo
