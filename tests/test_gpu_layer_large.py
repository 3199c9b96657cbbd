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


def test_append_of_many_blocks():
    """2^28 + 21 new tokens of one sequence, of which a few blocks are held."""
    import numpy as np
    from tests import kv8_ref
    bs, dim, n = 16, 64, (1 << 28) + 21
    width = -(-n // bs)
    places = [0, (1 << 23) - 1, 1 << 23, (1 << 24) - 1, 1 << 24, width - 1]
    x = torch.zeros(n, 1, dim, dtype=torch.bfloat16, device="cuda")
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    cache = q.KV8Cache.empty(len(places), 1, dim, bs)
    rng = np.random.default_rng(1)
    rows = {}
    for i, p in enumerate(places):
        m = min(bs, n - p * bs)
        rows[i] = torch.from_numpy(rng.standard_normal((m, 1, dim)).astype(np.float32)).bfloat16()
        x[p * bs:p * bs + m] = rows[i].cuda()
        table[0, p] = i
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qgemm_kv8_append(cache, x, x, table, i32(0, n), i32(n), n)
    for i, row in rows.items():
        m = row.shape[0]
        ref = {"k": torch.zeros(1, 1, bs, dim, dtype=torch.float8_e4m3fn),
               "v": torch.zeros(1, 1, dim, bs, dtype=torch.float8_e4m3fn), "k_scale": torch.zeros(1, 1),
               "v_scale": torch.zeros(1, 1)}
        kv8_ref.append(ref, row, row, [[0]], [0, m], [m], "e4m3")
        assert torch.equal(bits(cache.k[i, :, :m]).cpu(), bits(ref["k"][0, :, :m])), places[i]
        assert torch.equal(bits(cache.v[i, :, :, :m]).cpu(), bits(ref["v"][0, :, :, :m])), places[i]
        assert torch.equal(cache.k_scale[i].cpu(), ref["k_scale"][0]) and torch.equal(cache.v_scale[i].cpu(), ref["v_scale"][0])
