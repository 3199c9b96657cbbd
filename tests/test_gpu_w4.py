"""GPU tests of the 4-bit matvec against the formula in 64 bits: row counts
through every variant, odd N, K that ends inside a 128-weight chunk, groups,
zero points, both MX scale layouts, strides, bias, another stream and graphs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6])


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _make(kind, M, N, K, group, zeros, seed, bias=False, srows=1):
    rng = np.random.default_rng(seed)
    d = {"x": torch.from_numpy(rng.standard_normal((M, K)).astype(np.float32)).bfloat16(),
         "w": torch.from_numpy(rng.integers(0, 256, (N, K // 2), dtype=np.uint8)),
         "zeros": None, "bias": None}
    if kind == "mx":
        d["scales"] = torch.from_numpy(rng.integers(100, 140, (-(-N // srows), K // 32), dtype=np.uint8))
    else:
        d["scales"] = torch.from_numpy(rng.uniform(-0.02, 0.05, (N, K // group)).astype(np.float32)).bfloat16()
        if zeros:
            d["zeros"] = torch.from_numpy(rng.integers(0, 16, (N, K // group), dtype=np.uint8))
    if bias:
        d["bias"] = torch.from_numpy(rng.standard_normal(N).astype(np.float32) * 5).bfloat16()
    return d


def _want(kind, d, group, srows=1):
    """(result, allowed error) in 64 bits.  bf16 of the result (2^-8 relative);
    binary32 sums: of 128 + w (at most 143) for int4 with the zero point's part
    taken off again, K terms at the worst in one chain of K/8/32 products of
    32 (any order inside): (K/8 + 64) units of 2^-24 of the summed magnitudes."""
    x = d["x"].double().numpy()
    w = d["w"].numpy()
    nib = np.stack([w & 15, w >> 4], 2).reshape(w.shape[0], -1)
    N, K = nib.shape
    if kind == "mx":
        s = np.repeat(np.repeat(2.0 ** (d["scales"].numpy().astype(np.float64) - 127), srows, 0)[:N], 32, 1)
        v = E2M1[nib] * s
        size = np.abs(v)
    else:
        s = np.repeat(d["scales"].double().numpy(), group, 1)
        z = 8.0 if d["zeros"] is None else np.repeat(d["zeros"].numpy().astype(np.float64), group, 1)
        v = (nib - z) * s
        size = (143.0 + 128.0 + 15.0) * np.abs(s)
    y = x @ v.T
    tol = (K / 8 + 64) * 2.0 ** -24 * (np.abs(x) @ size.T)
    if d["bias"] is not None:
        b = d["bias"].double().numpy()
        y = y + b
        tol = tol + 2.0 ** -23 * np.abs(b)
    return y, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(y) + 2.0 ** -133


def _run(kind, d, b_layout=1, **kw):
    t = {n: (v.cuda() if v is not None else None) for n, v in d.items()}
    if kind == "mx":
        return q.qgemm_w4_matvec_mx(t["x"], t["w"], t["scales"], b_layout, bias=t["bias"], **kw)
    return q.qgemm_w4_matvec_i4(t["x"], t["w"], t["scales"], t["zeros"], bias=t["bias"], **kw)


def _check(out, want, tol):
    off = np.abs(out.double().cpu().numpy() - want) - tol
    assert off.max() <= 0, (off.max(), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("kind,group", [("i4", 32), ("i4", 64), ("i4", 128), ("mx", 32)])
@pytest.mark.parametrize("M", [1, 2, 4, 5, 16, 17, 32, 33, 64])
def test_rows(kind, group, M):
    for N, K in ((1, group), (17, 3 * group), (100, 1920 if group == 128 else 1984), (48, 8192)):
        for zeros in ((False, True) if kind == "i4" else (False,)):
            d = _make(kind, M, N, K, group, zeros, M + N + K, bias=zeros)
            _check(_run(kind, d), *_want(kind, d, group))


@pytest.mark.parametrize("K", [32, 64, 96, 128, 160, 1056])
@pytest.mark.parametrize("kind", ["i4", "mx"])
def test_ends_inside_a_chunk(kind, K):
    d = _make(kind, 3, 40, K, 32, kind == "i4", K)
    _check(_run(kind, d), *_want(kind, d, 32))


@pytest.mark.parametrize("N", [31, 32, 33, 200])
def test_mx_scales_of_32_rows(N):
    d = _make("mx", 2, N, 512, 32, False, N, bias=True, srows=32)
    _check(_run("mx", d, 32), *_want("mx", d, 32, 32))


def test_mx_scale_codes_at_the_ends():
    d = _make("mx", 1, 64, 128, 32, False, 1)
    d["scales"][:16] = 0
    d["scales"][16:32] = 1
    d["scales"][32:48] = 251
    d["x"] *= 2.0 ** -10
    d["scales"][48] = 255
    out = _run("mx", d)
    assert bool(out[:, 48].isnan().all())
    y, tol = _want("mx", d, 32)
    keep = np.arange(64) != 48
    _check(out[:, keep], y[:, keep], tol[:, keep])


def test_strides_bias_and_untouched_columns():
    d = _make("i4", 5, 50, 256, 64, True, 4, bias=True)
    x = torch.zeros(5, 256 + 24, dtype=torch.bfloat16)
    x[:, :256] = d["x"]
    w = torch.full((50, 128 + 48), 255, dtype=torch.uint8)
    w[:, :128] = d["w"]
    buf = torch.full((5, 61), 3.0, dtype=torch.bfloat16, device="cuda")
    out = q.qgemm_w4_matvec_i4(x.cuda()[:, :256], w.cuda()[:, :128], d["scales"].cuda(), d["zeros"].cuda(),
                               bias=d["bias"].cuda(), out=buf[:, :50])
    _check(out, *_want("i4", d, 64))
    assert bool((buf[:, 50:] == 3.0).all())


def test_matches_the_mx_gemm():
    """The same MXFP4 weights through qgemm_mx_mixed, with activations that
    e4m3 holds exactly."""
    rng = np.random.default_rng(5)
    d = _make("mx", 16, 96, 512, 32, False, 5)
    codes = torch.from_numpy(rng.integers(-8, 9, (16, 512)).astype(np.float32))
    d["x"] = codes.bfloat16()
    a = codes.cuda().to(torch.float8_e4m3fn).view(torch.uint8)
    sa = torch.full((16, 16), 127, dtype=torch.uint8, device="cuda")
    gemm = q.qgemm_mx_mixed(q.QGEMM_MX_E4M3, q.QGEMM_MX_E2M1, a, d["w"].cuda(), sa, d["scales"].cuda(), 1)
    y, tol = _want("mx", d, 32)
    out = _run("mx", d)
    _check(out, y, tol)
    assert (np.abs(gemm.double().cpu().numpy() - out.double().cpu().numpy()) <= 2 * tol).all()


@pytest.mark.parametrize("kind", ["i4", "mx"])
def test_another_stream_and_graph(kind):
    d = _make(kind, 4, 700, 2048, 32, False, 9)
    t = {n: v.cuda() for n, v in d.items() if v is not None}
    out = torch.empty(4, 700, dtype=torch.bfloat16, device="cuda")

    def call(**kw):
        if kind == "mx":
            return q.qgemm_w4_matvec_mx(t["x"], t["w"], t["scales"], 1, **kw)
        return q.qgemm_w4_matvec_i4(t["x"], t["w"], t["scales"], **kw)
    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = call()
    side.synchronize()
    assert torch.equal(want.view(torch.int16), again.view(torch.int16))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    for _ in range(3):
        t["x"].mul_(0.5)
        want = call()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want.view(torch.int16), out.view(torch.int16))


def test_python_refusals():
    d = _make("i4", 2, 32, 256, 64, True, 1)
    x, w, s, z = (d[n].cuda() for n in ("x", "w", "scales", "zeros"))
    for args in ((x[:, :128], w, s, z), (x.float(), w, s, z), (x, w, s.float(), z), (x, w, s[:, :3].contiguous(), z),
                 (x, w, s, z[:16]), (x, w, s, z.int()), (x.repeat(33, 1), w, s, z)):
        with pytest.raises(ValueError):
            q.qgemm_w4_matvec_i4(*args)
    with pytest.raises(ValueError):
        q.qgemm_w4_matvec_mx(x, w, z, 1)
    with pytest.raises(ValueError):
        q.qgemm_w4_matvec_mx(x, w, torch.zeros(32, 8, dtype=torch.uint8, device="cuda"), 16)
    with pytest.raises(ValueError):
        q.qgemm_w4_matvec_i4(x, w, s, z, out=torch.empty(2, 31, dtype=torch.bfloat16, device="cuda"))
