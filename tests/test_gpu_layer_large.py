"""GPU tests of the decoder-layer operators where one launch cannot hold all
threads (2^32): the parts' first and last rows against calls on those rows
alone."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.empty_cache()


def bits(t):
    return t.contiguous().view(torch.uint8)


@pytest.mark.parametrize("kind", ["i8", "f8", "mx8", "mx4"])
def test_norm_of_many_rows(kind):
    from tests.test_gpu_rmsnorm import _call
    M, K = (1 << 24) + 5, 32
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(M, K, device="cuda", generator=g, dtype=torch.bfloat16)
    r = torch.randn(M, K, device="cuda", generator=g, dtype=torch.bfloat16)
    gamma = torch.randn(K, device="cuda", generator=g).bfloat16()
    got = _call(kind, x, gamma, residual=r)
    for lo in (0, (1 << 23) - 3, (1 << 24) - 3):
        hi = min(lo + 8, M)
        want = _call(kind, x[lo:hi].contiguous(), gamma, residual=r[lo:hi].contiguous())
        for a, b in zip(got, want):
            assert torch.equal(bits(a[lo:hi]), bits(b)), lo
