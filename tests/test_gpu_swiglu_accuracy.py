"""GPU tests of how near SwiGLU's values are to the formula in 64 bits: gates far
below zero, where silu is as small as exp(g), down to the end of binary32's
range, and the scales and codes that follow from them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

from tests.test_gpu_rmsnorm import KINDS  # noqa: E402
from tests.test_gpu_swiglu import call, check_codes  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# With a = exp(-|g|), silu u = g a / (1 + a) u: exp2 to a unit in the last place
# (2 in units of 2^-24) of an argument below a half (0.2 more), which 1 + a
# takes part of the other way; then the sum, the reciprocal, three products (1
# each): 7.2.
REL = 8 * 2.0 ** -24
# a itself below binary32's normal range: half a step, 2^-150, or, past
# |g| = 104, a zero for less than that; times |g| <= 104
ABS = 2.0 ** -143 + 2.0 ** -149
Q_TOL = 4 * 2.0 ** -24           # the scale, its reciprocal, the quotient


def formula(x):
    g, u = (t.numpy().astype(np.longdouble) for t in x.double().cpu().chunk(2, 1))
    with np.errstate(over="ignore"):
        return (g / (1 + np.exp(-g)) * u).astype(np.float64), np.abs(u).astype(np.float64)


def check(kind, x, tol=Q_TOL):
    y, u = formula(x)
    codes, scale = call(kind, x)
    check_codes(kind, y, np.abs(y) * REL + u * ABS + 2.0 ** -149, codes, scale, tol)
    return codes, scale


def gates(M, I, lo, hi, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(M, 2 * I, device="cuda", generator=g)
    x[:, :I] = lo + (hi - lo) * torch.rand(M, I, device="cuda", generator=g)
    return x.bfloat16()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lo,hi", [(-35, -5), (-60, -30), (-80, -35), (-87, -75)])
@pytest.mark.parametrize("M,I", [(3, 1024), (400, 2176), (2, 8192 + 256)])
def test_gates_far_below_zero(kind, lo, hi, M, I):
    x = gates(M, I, lo, hi, M)
    x[:, I:] += torch.sign(x[:, I:])                     # no up value so small that the product is out of range
    _, scale = check(kind, x)
    assert bool((scale != 0).any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lo,hi,up", [(-88.5, -87, 2.0 ** 60), (-92, -88, 2.0 ** 90), (-100, -87, 2.0 ** 120)])
def test_gates_at_the_end_of_the_range(kind, lo, hi, up):
    """exp(-|g|) is below binary32's normal range, the product with a large up
    value is not."""
    x = gates(8, 512, lo, hi, 7)
    x[:, 512:] = torch.sign(x[:, 512:]) * up
    codes, scale = check(kind, x)
    assert bool((scale != 0).all()) and bool((codes.view(torch.uint8) & 0x77 != 0).any())


@pytest.mark.parametrize("kind", KINDS)
def test_every_gate(kind):
    """All finite bf16 gates, alone in their blocks with one up value."""
    g = torch.arange(0, 0x7f80, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    for gate in (g, -g):
        x = torch.zeros(g.numel(), 256, dtype=torch.bfloat16, device="cuda")
        x[:, 3], x[:, 128 + 3] = gate, 0.75
        check(kind, x)


@pytest.mark.parametrize("kind", ["i8", "f8", "block"])
def test_quotients_are_the_divided_ones(kind):
    """Rows of whole scales s and values s c, c half way between two codes: a
    quotient that is a unit in the last place off takes the odd one."""
    s = torch.arange(33, 256, 2, device="cuda").float()              # (silu is its gate itself)
    if kind == "i8":
        c, top = torch.arange(127, device="cuda") + 0.5, 127.0
        want = torch.round(c)                                        # ties to even
    else:
        c = torch.cat([torch.arange(17, 32, 2, device="cuda") * 2.0 ** i for i in range(-6, 4)])
        top, want = 448.0, c.to(torch.float8_e4m3fn).float()
    I = 128
    x = torch.zeros(s.numel(), 2 * I, device="cuda")
    x[:, :I] = s[:, None]
    x[:, I], x[:, I + 1:I + 1 + c.numel()] = top, c
    assert torch.equal(x, x.bfloat16().float())
    codes, scale = call(kind, x.bfloat16())
    assert torch.equal(scale.view(-1), s)
    got = (codes if kind == "i8" else codes.view(torch.float8_e4m3fn)).float()
    assert bool((got[:, 0] == top).all()) and torch.equal(got[:, 1:1 + c.numel()], want.expand(s.numel(), -1))
