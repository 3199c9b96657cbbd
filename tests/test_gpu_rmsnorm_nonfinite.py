"""GPU tests of the RMS norm with quantised output on rows that hold what is
not a number: their scales say so, the GEMM's row is NaN, other rows keep their
bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

from tests.test_gpu_rmsnorm import KINDS, _call, _data  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def gemm(kind, codes, scale, K):
    """The rows times a weight of ones."""
    w = torch.ones(32, K, device="cuda").bfloat16()
    one = torch.ones(32, device="cuda")
    if kind == "i8":
        return q.qgemm_i8_rowwise(codes, torch.ones(32, K, dtype=torch.int8, device="cuda"), scale, one)
    if kind == "f8":
        return q.qgemm_f8_pertoken(codes, *(lambda c, s: (c, scale, s))(*q.qgemm_quant_f8_pertoken(w)))
    if kind == "block":
        wq = torch.ones(128, K, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        return q.qgemm_f8_blockscale(codes, wq, scale, torch.ones(1, K // 128, device="cuda"))
    fmt = q.QGEMM_MX_E4M3 if kind == "mx8" else q.QGEMM_MX_E2M1
    wq, ws = q.qgemm_quant_mx(fmt, w)
    return q.qgemm_mx(fmt, codes, wq, scale, ws, 1)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("K", [256, 4096, 16384 + 2048])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("where", ["x", "residual", "gamma 0"])
def test_shows_in_the_scales(kind, K, bad, where):
    x, r, gamma = _data(7, K, K)
    at, row = K - 70, 3
    if where == "gamma 0":
        gamma[at] = 0
    want, ws, wr = _call(kind, x, gamma, residual=r)
    (r if where == "residual" else x)[row, at] = bad
    codes, scale, total = _call(kind, x, gamma, residual=r)
    keep = torch.arange(7, device="cuda") != row
    assert torch.equal(codes[keep], want[keep]) and torch.equal(scale[keep], ws[keep])
    total[row, at] = wr[row, at]
    assert torch.equal(total.view(torch.int16), wr.view(torch.int16))     # the sum itself is bf16(x + r)
    s = scale[row].flatten()
    if kind in ("block", "mx8", "mx4"):
        own = at // (128 if kind == "block" else 32)
        s = s if bad != bad else s[own:own + 1]
    assert bool((s == 255).all() if kind.startswith("mx") else s.isnan().all())
    out = gemm(kind, codes, scale, K)
    assert bool(out[row].isnan().all()) and bool(out[keep].isfinite().all())


@pytest.mark.parametrize("kind", KINDS)
def test_sums_past_binary32_give_zeros(kind):
    x, r, gamma = _data(3, 512, 1)
    x[1] = 2.0 ** 70
    codes, scale, _ = _call(kind, x, gamma, residual=r)
    assert not bool(scale[1].any()) and not bool((codes[1] & (0x7F if kind != "mx4" else 0x77)).any())
