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


@pytest.mark.parametrize("kind", ["i8", "f8", "block", "mx8", "mx4"])
def test_norm_of_many_rows(kind):
    from tests.test_gpu_rmsnorm import _call
    M, K = (1 << 24) + 5, 128 if kind == "block" else 32
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


@pytest.mark.parametrize("kind,srows,M", [("mx", 1, 2), ("mx", 32, 1), ("i4", 1, 1), ("i4", 1, 17)])
def test_matvec_of_many_weight_rows(kind, srows, M):
    from tests.test_gpu_w4_exact import make, run, want
    N, K = (1 << 27) + 37, 32
    d = make(kind, M, N, K, 32, 1, kind == "i4", True, srows)
    got = run(kind, d, srows)
    for lo in (0, (1 << 26) - 64, (1 << 27) - 64):
        hi = min(lo + 128, N)
        part = dict(d, w=d["w"][lo:hi], bias=d["bias"][lo:hi], scales=d["scales"][lo // srows:-(-hi // srows)],
                    zeros=None if d["zeros"] is None else d["zeros"][lo:hi])
        assert torch.equal(got[:, lo:hi], want(kind, part, 32, srows).bfloat16()), lo
