"""GPU tests of what the operators of a layer of experts refuse by its shape:
arrays of the right length whose rows are not the tokens' choices, by the
compiled binding and by the full way."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402
from block_scaled_precision_02_amd import experts, layer  # noqa: E402

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


@pytest.mark.parametrize("shape", [(3, 7), (21,), (1, 21), (21, 1), (7, 3, 1)])
def test_one_value_for_each_choice(way, shape):
    position, w, x, y, r = data(7, 3, 8, 64, 1)
    bad = torch.zeros(shape, device="cuda")
    for call in (lambda: q.qgemm_moe_combine(y, position, bad), lambda: q.qgemm_moe_combine(y, position, bad, residual=r),
                 lambda: q.qgemm_moe_combine_grad(r, y, position, bad),
                 lambda: q.qgemm_moe_combine_grad(r, y, position, w, dweights=bad)):
        with pytest.raises(ValueError):
            call()
    dw = torch.zeros(7, 3, device="cuda")
    assert q.qgemm_moe_combine_grad(r, y, position, w, dweights=dw)[1] is dw


@pytest.mark.parametrize("kw", [dict(position=(3, 7)), dict(position=(21,)), dict(order=(7, 3)), dict(order=(21, 1)),
                                dict(offsets=(3, 3)), dict(offsets=(1, 9))])
def test_the_sort_writes_what_the_others_read(way, kw):
    position, *_ = data(7, 3, 8, 64, 1)
    ids = position.clamp(-1, 7).contiguous()
    out = {n: torch.zeros(s, dtype=torch.int32, device="cuda") for n, s in kw.items()}
    with pytest.raises(ValueError):
        q.qgemm_moe_sort(ids, 8, **out)
