"""GPU tests of grouped GEMMs without columns or rows, and of numbers of rows that
are none, by the compiled binding and by the full way."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402
from block_scaled_precision_02_amd import experts, layer  # noqa: E402

from tests.test_gpu_grouped import KINDS, Case  # noqa: E402
from tests.test_gpu_moe import data  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture(params=["compiled", "full"])
def way(request, monkeypatch):
    assert layer._fast is not None, "_fast.so is not built"
    if request.param == "full":
        for m in (layer, experts):
            monkeypatch.setattr(m, "_fast", None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,top_k", [([3, 0, 5], 0), ([3, 0, 5], 2), ([4], 0), ([0, 0], 0)])
def test_no_columns(way, kind, counts, top_k):
    c = Case(kind, counts, 0, 256, top_k)
    assert tuple(c.b.shape[:2]) == (len(counts), 0)
    out = c.call()
    assert tuple(out.shape) == (sum(counts), 0) and out.dtype == torch.bfloat16
    given = torch.empty(sum(counts), 0, dtype=torch.bfloat16, device="cuda")
    assert c.call(out=given) is given


@pytest.mark.parametrize("rows", [-1, -2 ** 40, 1 << 31, 1 << 70, 2.5, "x", [3], float("nan")])
def test_gather_rows_that_are_no_number_of_rows(way, rows):
    position, w, x, y, r = data(7, 3, 8, 64, 1)
    with pytest.raises(ValueError):
        q.qgemm_moe_gather(x, position, rows=rows)
    with pytest.raises(ValueError):
        q.qgemm_moe_gather(x, position, rows=rows, out=y)


def test_gather_into_no_rows(way):
    position, w, x, y, r = data(7, 3, 8, 64, 1)
    assert q.qgemm_moe_gather(x, position, rows=0).shape == (0, 64)
    assert q.qgemm_moe_gather(x, position, rows=21, out=y) is y
