"""The grouped GEMMs against the conservative-sync twin of the library (every
wait drained, a barrier at every stage boundary): the same bits, so no wait is
miscounted.  Every LDS-staged tile, K with whole and partial last rounds."""
import ctypes
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402
from block_scaled_precision_02_amd import build  # noqa: E402

from tests.test_gpu_grouped import KINDS, Case, spread  # noqa: E402


@pytest.fixture(scope="module")
def twin():
    if not os.path.exists(build.LIB_SYNC):
        pytest.fail(f"{build.LIB_SYNC} is not built (python -m block_scaled_precision_02_amd.build)")
    return q.declare(ctypes.CDLL(build.LIB_SYNC))


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,experts,N,K", [
    (300, 64, 1040, 128), (300, 64, 1040, 1408), (500, 70, 1200, 4096),     # panels
    (700, 12, 400, 1664), (900, 16, 260, 384),                             # 128x128
    (900, 16, 3700, 1664), (1500, 32, 2049, 256), (2000, 60, 1025, 2304),  # 128x256
    (3000, 12, 520, 1408), (2500, 5, 300, 2048),                           # 256x256
    (9000, 3, 264, 896)])                                                  # blockscale's 256x128
def test_fast_build_equals_sync_twin(twin, monkeypatch, kind, rows, experts, N, K):
    c = Case(kind, spread(rows, experts, N + K), N, K, 2, bias=True, seed=rows)
    fast = q.lib()
    for _ in range(3):
        a = c.call()
        monkeypatch.setattr(q, "_lib", twin)
        b = c.call()
        torch.cuda.synchronize()
        monkeypatch.setattr(q, "_lib", fast)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
