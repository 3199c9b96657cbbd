"""GPU tests of the decoder-layer operators on a given stream: what they
allocate for themselves is not memory that the current stream's earlier work
still uses, nor is it handed out again before both streams have used it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

from tests.test_gpu_kv8 import Setup  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def calls():
    """name -> (call(stream), bytes of what it allocates)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x = torch.randn(64, 4096, device="cuda", generator=g).bfloat16()
    gamma = torch.ones(4096, device="cuda").bfloat16()
    w = torch.randint(0, 256, (8192, 2048), dtype=torch.uint8, device="cuda", generator=g)
    s1 = torch.full((8192, 128), 120, dtype=torch.uint8, device="cuda")
    s4 = torch.ones(8192, 32, device="cuda").bfloat16()
    s = Setup("e4m3", 1, 128, 64, [(1, 9000)], seed=15)
    cache, Q = s.gpu(), s.bf16(1, 4, 128).cuda()
    args = s.seqs() + (1, 9000)
    need = q.lib().qgemm_kv8_attention_workspace(cache._ref, 1, 1, 4, 1, 9000, 1, 0)
    assert need > 0
    out = torch.empty_like(Q)
    return {
        "i8": (lambda st: q.qgemm_rmsnorm_quant_i8_rowwise(x, gamma, residual=x, stream=st), (64 * 4096, 256, 64 * 8192)),
        "f8": (lambda st: q.qgemm_rmsnorm_quant_f8_pertoken(x, gamma, residual=x, stream=st), (64 * 4096, 256, 64 * 8192)),
        "block": (lambda st: q.qgemm_rmsnorm_quant_f8_block(x, gamma, residual=x, stream=st), (64 * 4096, 64 * 128, 64 * 8192)),
        "mx": (lambda st: q.qgemm_rmsnorm_quant_mx(0, x, gamma, residual=x, stream=st), (64 * 4096, 64 * 128, 64 * 8192)),
        "w4 mx": (lambda st: q.qgemm_w4_matvec_mx(x, w, s1, 1, stream=st), (64 * 8192 * 2,)),
        "w4 i4": (lambda st: q.qgemm_w4_matvec_i4(x, w, s4, stream=st), (64 * 8192 * 2,)),
        "attention": (lambda st: q.qgemm_kv8_attention(cache, Q, *args, stream=st), (1024, need)),
        "workspace": (lambda st: q.qgemm_kv8_attention(cache, Q, *args, out=out, stream=st), (need,)),
    }


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", ["i8", "f8", "block", "mx", "w4 mx", "w4 i4", "attention", "workspace"])
def test_new_memory_is_not_in_use_elsewhere(name, raw):
    """The current stream still has to read memory that was let go; the call on
    the other stream, which starts at once, must not get it."""
    call, sizes = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    held = [torch.full((n,), 90 + i, dtype=torch.uint8, device="cuda") for i, n in enumerate(sizes)]
    keep = [torch.empty_like(t) for t in held]
    torch.cuda.synchronize()
    for _ in range(100):
        big = big * 1.0001
    for k, t in zip(keep, held):
        k.copy_(t)
    del held, t
    got = call(side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    for i, k in enumerate(keep):
        assert bool((k == 90 + i).all())
    for a, b in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, want))):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("name", ["f8", "w4 mx", "attention"])
def test_results_let_go_are_kept_for_the_current_stream(name):
    """A result that the current stream still has to read, let go and followed
    by another call on the other stream."""
    call, _ = calls()[name]
    first = lambda v: v[0] if isinstance(v, tuple) else v  # noqa: E731
    want = first(call(None))
    side = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    got = first(call(side))
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(100):
        big = big * 1.0001
    keep = got.clone()
    n = got.numel() * got.element_size()
    del got
    with torch.cuda.stream(side):
        torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert torch.equal(keep.view(torch.uint8), want.view(torch.uint8))


def test_the_default_stream_by_its_handle():
    call, _ = calls()["w4 mx"]
    want = call(None)
    assert torch.equal(call(torch.cuda.default_stream()), want)
    assert torch.equal(call(torch.cuda.default_stream().cuda_stream), want)
