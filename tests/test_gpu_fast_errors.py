"""GPU tests of how the compiled binding of the expert operators fails: a launch
error is raised at once, and the call is not made a second time."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402
from block_scaled_precision_02_amd import experts, layer  # noqa: E402

from tests.test_gpu_fast_binding import NAMES, calls  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("name", NAMES)
def test_a_launch_error_is_raised_once(name, monkeypatch):
    assert layer._fast is not None, "_fast.so is not built"
    call = calls()[name]
    call()

    def again(*a):
        raise AssertionError("the call was made again")
    for m in (layer, experts):
        monkeypatch.setattr(m, "_enqueue", again)
    monkeypatch.setenv("QGEMM_INJECT_LAUNCH_ERROR", "719")
    for _ in range(2):
        with pytest.raises(q.QGemmError, match="injected error 719") as e:
            call()
        assert e.value.status == q.QGEMM_ERR_HIP and not isinstance(e.value, ValueError)
    monkeypatch.delenv("QGEMM_INJECT_LAUNCH_ERROR")
    call()
