"""GPU tests of the grouped GEMMs: int8 against the exact sum and the epilogue's
roundings by equality, the other paths against 64 bits within the roundings of
a binary32 sum and of the result; every tile, rows by an order and rows as they
are, experts without rows, with one row and with most of them, odd columns,
bias, strides, rows behind the last one, broken offsets, streams, graphs."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

KINDS = ["i8", "f8", "block", "mx8", "mx4"]
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Case:
    """counts: rows of each expert; extra: room behind the last one; top_k > 0:
    A holds tokens and an order (not of a sort: any tokens, in any order)."""

    def __init__(self, kind, counts, N, K, top_k=0, bias=False, extra=0, seed=0):
        self.kind, self.counts, self.N, self.K, self.top_k = kind, counts, N, K, top_k
        self.E, live = len(counts), sum(counts)
        self.rows = live + extra
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def ints(lo, hi, *s, dtype=torch.uint8):
            return torch.randint(lo, hi, s, device="cuda", generator=g, dtype=dtype)

        def rand(*s):
            return torch.rand(*s, device="cuda", generator=g)
        self.offsets = torch.tensor(np.cumsum([0] + list(counts)), dtype=torch.int32, device="cuda")
        m = self.rows
        self.order = None
        if top_k:
            m = max(1, -(-self.rows // top_k))
            self.order = ints(0, m * top_k, self.rows, dtype=torch.int32)
            self.order[live:] = -1
        self.m = m

        def codes(*s):
            if kind == "i8":
                return ints(-127, 128, *s, dtype=torch.int8)
            if kind == "mx4":
                return ints(0, 256, *s[:-1], s[-1] // 2)
            return (torch.randn(*s, device="cuda", generator=g) * 60).clamp(-448, 448).to(
                torch.float8_e4m3fn).view(torch.uint8)
        self.a, self.b = codes(m, K), codes(self.E, N, K)
        if kind in ("i8", "f8"):
            self.sa, self.sb = 0.5 + rand(m), 0.01 + 0.01 * rand(self.E, N)
        elif kind == "block":
            self.sa, self.sb = 0.5 + rand(m, K // 128), 0.01 + 0.01 * rand(self.E, -(-N // 128), K // 128)
        else:
            self.sa, self.sb = ints(120, 130, m, K // 32), ints(118, 126, self.E, N, K // 32)
        self.bias = torch.randn(self.E, N, device="cuda", generator=g).bfloat16() if bias else None

    def call(self, **kw):
        args = [self.a, self.b, self.sa, self.sb, self.offsets]
        kw = dict(dict(order=self.order, top_k=self.top_k or 1, bias=self.bias), **kw)
        if self.kind.startswith("mx"):
            return q.qgemm_mx_grouped(q.QGEMM_MX_E4M3 if self.kind == "mx8" else q.QGEMM_MX_E2M1, *args, **kw)
        f = {"i8": q.qgemm_i8_rowwise_grouped, "f8": q.qgemm_f8_pertoken_grouped,
             "block": q.qgemm_f8_blockscale_grouped}[self.kind]
        return f(*args, **kw)

    def _wide(self, codes, scales, per):
        """float64 values; per: rows a scale row covers."""
        if self.kind == "i8":
            return codes.double()
        if self.kind == "mx4":
            v = torch.tensor(E2M1, dtype=torch.float64, device="cuda")[
                torch.stack([codes & 15, codes >> 4], 2).long()].view(codes.shape[0], self.K)
        else:
            v = codes.view(torch.float8_e4m3fn).double()
        if self.kind == "f8":
            return v * scales.double()[:, None]
        s = scales.double() if self.kind == "block" else torch.exp2(scales.double() - 127)
        s = s.repeat_interleave(per, 0)[:codes.shape[0]]
        return v * s.repeat_interleave(128 if self.kind == "block" else 32, 1)

    def check(self, out):
        at = 0
        for e, n in enumerate(self.counts):
            if n == 0:
                continue
            rows = torch.arange(at, at + n, device="cuda")
            if self.order is not None:
                rows = self.order[rows].long() // self.top_k
            a = self._wide(self.a[rows], self.sa[rows], 1)
            b = self._wide(self.b[e], self.sb[e], 128 if self.kind == "block" else 1)
            got = out[at:at + n]
            sums = torch.mm(a, b.t().contiguous())
            if self.kind == "i8":
                # the exact sum, then the epilogue's own roundings one by one
                f = sums.float() * self.sa[rows][:, None]
                f = f * self.sb[e][None, :]
                if self.bias is not None:
                    f = f + self.bias[e].float()[None, :]
                assert torch.equal(got.view(torch.int16), f.bfloat16().view(torch.int16)), e
            else:
                size = torch.mm(a.abs(), b.abs().t().contiguous())
                want = sums
                if self.bias is not None:
                    want = want + self.bias[e].double()[None, :]
                    size = size + self.bias[e].double().abs()[None, :]
                # the library's own bound for these products (tests/parity.py): the matrix
                # cores align the products of one instruction to their largest before they
                # add them.  The tests of equality below hold them to the bit.
                assert bool(((got.double() - want).abs() <= 1e-2 * size + 2.0 ** -7 * want.abs()).all()), e
            at += n


def spread(total, experts, seed):
    """Uneven counts that sum to total."""
    rng = np.random.default_rng(seed)
    return np.bincount(rng.choice(experts, total, p=(w := rng.random(experts) ** 3) / w.sum()), minlength=experts).tolist()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,N,K", [
    ([1], 16, 128), ([0, 1, 0], 40, 256), ([3, 0, 17, 16, 1], 130, 384),
    ([20, 0, 0, 129, 300, 1], 200, 640),                              # 128x128 tiles
    ([513, 0, 256, 1, 700], 300, 512),                                # 256-row tiles
    ([5000, 1, 3200], 200, 256),                                      # blockscale's
    ([300, 64, 130, 192, 65], 264, 768),                              # waves with half their rows, and none
    ([1] * 100, 64, 1152), ([0] * 30 + [40] + [0] * 33, 256, 2048)])
@pytest.mark.parametrize("top_k", [0, 3])
def test_sizes(kind, counts, N, K, top_k):
    c = Case(kind, counts, N, K, top_k, bias=len(counts) % 2 == 0, seed=N + K)
    c.check(c.call())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,N,K", [
    ([20, 0, 129, 1, 64, 65, 128, 0, 17, 33, 96, 40, 0, 2, 100, 31], 3801, 256),    # 15 columns of tiles, the last in part
    ([0, 300] + [0] * 6 + [1] * 100 + [40, 90, 128, 257], 513, 640),
    ([130] * 8 + [1], 4097, 1152)])
@pytest.mark.parametrize("top_k", [0, 3])
def test_tiles_of_256_columns(kind, counts, N, K, top_k):
    c = Case(kind, counts, N, K, top_k, bias=top_k == 3, extra=top_k, seed=N + K)
    out = torch.full((c.rows, N + (-N) % 8), 9.0, dtype=torch.bfloat16, device="cuda")
    c.call(out=out[:, :N])
    c.check(out[:, :N])
    assert bool((out[:, N:] == 9).all()) and bool((out[sum(counts):] == 9).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,experts,N,K", [(60, 200, 272, 256), (500, 70, 136, 896), (3000, 24, 520, 384),
                                              (5000, 12, 264, 1280), (900, 1, 1024, 256), (2000, 1024, 48, 128),
                                              (300, 64, 1100, 640), (700, 60, 1161, 384)])
def test_uneven(kind, rows, experts, N, K):
    for top_k in (0, 8):
        c = Case(kind, spread(rows, experts, rows), N, K, top_k, seed=rows)
        c.check(c.call())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N", [1, 7, 31, 129, 257])
@pytest.mark.parametrize("each", [2, 90, 300])
def test_odd_columns(kind, N, each):
    c = Case(kind, [each, 1, each], N, 256, 2, bias=True, seed=N)
    c.check(c.call())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("experts,N", [(300, 129), (200, 385), (64, 1030), (7, 1537)])
def test_odd_columns_of_few_rows(kind, experts, N):
    """64-row panels and the stream of single waves."""
    for K in (128, 896):
        c = Case(kind, spread(2 * experts, experts, N), N, K, 2, bias=True, extra=3, seed=N)
        out = torch.full((c.rows, N + (-N) % 8), 9.0, dtype=torch.bfloat16, device="cuda")
        c.call(out=out[:, :N])
        c.check(out[:, :N])
        assert bool((out[:, N:] == 9).all()) and bool((out[2 * experts:] == 9).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("each", [5, 100, 260])
def test_rows_behind_the_last_and_strides(kind, each):
    c = Case(kind, [each, 0, each + 3], 200, 384, 2, extra=37, seed=each)
    buf = torch.full((c.rows + 1, 200 + 24), 9.0, dtype=torch.bfloat16, device="cuda")
    out = buf[:c.rows, 8:208]
    assert c.call(out=out) is out
    c.check(out)
    live = sum(c.counts)
    assert bool((buf[live:] == 9).all()) and bool((buf[:, :8] == 9).all()) and bool((buf[:, 208:] == 9).all())
    # rows of A in a wider buffer
    wide = torch.zeros(c.m, c.a.shape[1] + 32, dtype=c.a.dtype, device="cuda")
    wide[:, 16:16 + c.a.shape[1]] = c.a
    c.a = wide[:, 16:16 + c.a.shape[1]]
    assert torch.equal(c.call()[:live], out[:live])
    # and of B
    wide = torch.zeros(c.E, 200, c.b.shape[2] + 16, dtype=c.b.dtype, device="cuda")
    wide[:, :, :c.b.shape[2]] = c.b
    c.b = wide[:, :, :c.b.shape[2]]
    assert torch.equal(c.call()[:live], out[:live])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("each,N", [(4, 128), (80, 128), (280, 128), (4, 16384), (4, 4096), (80, 14352)])
def test_broken_offsets_and_orders_stay_in_range(kind, each, N):
    """Offsets outside the rows are clamped, tokens that are not there are zeros:
    nothing else is written."""
    c = Case(kind, [each] * 4, N, 256, 2, extra=10, seed=each)
    want = c.call()
    live = 4 * each
    c.order[3] = -1
    c.order[5 % each] = 2 ** 31 - 1
    got = c.call()
    keep = [i for i in range(live) if i not in (3, 5 % each)]
    assert torch.equal(got[keep], want[keep]) and not bool(got[3].any())
    good = c.offsets.clone()
    for values in ([-5, each, 2 * each, 3 * each, 10 ** 9], [0, 0, 0, 0, 0], [7, 3, 2, 1, 0], [2 ** 31 - 1] * 5,
                   [-2 ** 31] * 5):
        c.offsets = torch.tensor(values, dtype=torch.int32, device="cuda")
        buf = torch.full((c.rows + 64, N), 9.0, dtype=torch.bfloat16, device="cuda")
        c.call(out=buf[:c.rows])
        assert bool((buf[c.rows:] == 9).all())
        if values[0] == -5:
            assert torch.equal(buf[:live][keep], got[:live][keep])
        else:
            assert bool((buf == 9).all())
    c.offsets = good
    assert torch.equal(c.call()[keep], want[keep])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,N", [([70, 90, 100], 320), ([2, 70, 0, 13, 1] * 10, 1290), ([1, 3, 2], 2100),
                                      ([300, 200], 512)])
def test_a_row_has_the_same_bits_wherever_it_stands(kind, counts, N):
    """The sums' order is the sizes' alone: not the row's place, the expert's
    other rows, or the way its token is found."""
    c = Case(kind, counts, N, 512, 0, seed=8)
    out = c.call()
    assert torch.equal(out, c.call())
    back = torch.arange(c.rows, device="cuda").flip(0)
    c2 = Case(kind, counts[::-1], N, 512, 0, seed=8)
    c2.a, c2.sa, c2.b, c2.sb = c.a, c.sa, c.b.flip(0).contiguous(), c.sb.flip(0).contiguous()
    c2.order, c2.top_k = back.int().contiguous(), 1
    assert torch.equal(c2.call().flip(0), out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,N,K", [([1, 16, 5, 0, 40], 272, 384), ([90, 128, 0, 300, 1], 320, 640),
                                        ([700, 0, 255, 513], 520, 1152), ([40] * 8, 64, 128),
                                        ([300, 64, 130, 192, 65], 264, 768), ([5000, 1, 3200], 136, 256)])
def test_same_bits_as_the_dense_gemm(kind, counts, N, K):
    """Each expert's rows are those of the GEMM of the same name on one of its
    tiles."""
    c = Case(kind, counts, N, K, 3, bias=kind != "block", seed=N)
    out = c.call()
    at = 0
    for e, n in enumerate(counts):
        if not n:
            continue
        rows = c.order[at:at + n].long() // 3
        a, sa, bias = c.a[rows].contiguous(), c.sa[rows].contiguous(), c.bias[e] if c.bias is not None else None
        args, kw = (a, c.b[e], sa, c.sb[e].clone()), dict(bias=bias)
        if kind.startswith("mx"):
            def dense():
                return q.qgemm_mx(q.QGEMM_MX_E4M3 if kind == "mx8" else q.QGEMM_MX_E2M1, *args, 1, **kw)
        else:
            def dense():
                return {"i8": q.qgemm_i8_rowwise, "f8": q.qgemm_f8_pertoken, "block": q.qgemm_f8_blockscale}[kind](
                    *args, **kw)
        same = []
        for tile in (8, 7, 10 if kind == "block" else 5):
            q.force_tile(tile)
            try:
                same.append(torch.equal(dense().contiguous().view(torch.int16),
                                        out[at:at + n].contiguous().view(torch.int16)))
            finally:
                q.force_tile(-1)
        assert any(same), (e, same)
        at += n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts,N,K", [([3, 0, 17], 136, 896), ([100, 3, 250], 264, 640), ([600, 1, 300], 392, 512),
                                        (([30, 0, 1, 16] * 16), 1300, 640), ([5] * 9 + [0] * 20, 1312, 1152),
                                        ([1] * 8, 2056, 384)])
@pytest.mark.parametrize("top_k", [0, 2])
def test_exact_sums(kind, counts, N, K, top_k):
    """Small whole numbers under powers of two: every sum is exact in binary32,
    the result the formula's, rounded once."""
    c = Case(kind, counts, N, K, top_k, seed=K)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)

    def small(*s):
        return torch.randint(-4, 5, s, device="cuda", generator=g)
    if kind == "mx4":
        c.a, c.b = (torch.randint(0, 256, t.shape, device="cuda", generator=g, dtype=torch.uint8) & 0xbb
                    for t in (c.a, c.b))                     # magnitudes 0 to 1.5
    elif kind == "i8":
        c.a, c.b = small(*c.a.shape).to(torch.int8), small(*c.b.shape).to(torch.int8)
    else:
        c.a, c.b = (small(*t.shape).float().to(torch.float8_e4m3fn).view(torch.uint8) for t in (c.a, c.b))

    def power(t):
        if t.dtype == torch.uint8:
            return torch.randint(126, 128, t.shape, device="cuda", generator=g, dtype=torch.uint8)
        return torch.exp2(torch.randint(-1, 1, t.shape, device="cuda", generator=g).float())
    c.sa, c.sb = power(c.sa), power(c.sb)
    out, at = c.call(), 0
    for e, n in enumerate(counts):
        rows = torch.arange(at, at + n, device="cuda")
        if top_k:
            rows = c.order[rows].long() // top_k
        a, b = c._wide(c.a[rows], c.sa[rows], 1), c._wide(c.b[e], c.sb[e], 128 if kind == "block" else 1)
        if kind == "i8":
            a, b = a * c.sa[rows].double()[:, None], b * c.sb[e].double()[:, None]
        want = torch.mm(a, b.t().contiguous()).bfloat16()
        assert torch.equal(out[at:at + n].float(), want.float()), e
        at += n


@pytest.mark.parametrize("kind", KINDS)
def test_weights_past_4_gib(kind):
    N, K = 4096, 8192
    e = (5 << 30) // (N * K // (2 if kind == "mx4" else 1))
    counts = [0] * e
    counts[0] = counts[e // 2] = counts[-1] = 2
    c = Case(kind, counts, N, K, 0, seed=1)
    assert c.b.numel() > 1 << 32
    c.check(c.call())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("each,N", [(3, 256), (100, 256), (300, 256), (3, 4096), (3, 40000)])
def test_streams_and_graph(kind, each, N):
    c = Case(kind, [each, 2 * each], N, 256, 2, seed=2)
    want = c.call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.call(stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros(c.rows, N, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out=out)
    for i in range(3):
        # other tokens and other counts under the same graph
        c.order.copy_(c.order.roll(7))
        c.offsets.copy_(torch.tensor([0, min(each + 10 * i, 3 * each), 3 * each], dtype=torch.int32))
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c.call())


@pytest.mark.parametrize("kind", KINDS)
def test_empty_calls(kind):
    c = Case(kind, [0, 0, 0], 64, 128, 0)
    assert c.call().shape == (0, 64)
    c = Case(kind, [0, 0, 0], 64, 128, 2, extra=5)
    out = torch.full((5, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    c.call(out=out)
    assert bool((out == 9).all())


def test_top_k_from_the_order():
    c = Case("i8", [5, 3, 4], 64, 128, 3, seed=1)
    assert c.m == 4
    assert torch.equal(c.call(top_k=None), c.call())
    assert torch.equal(c.call(top_k=np.int64(3)), c.call())
    c.a, c.sa = torch.cat([c.a, c.a[:1]]), torch.cat([c.sa, c.sa[:1]])
    with pytest.raises(ValueError):
        c.call(top_k=None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("bad", [7, [1.0], "x"])
def test_refusals(kind, bad):
    c = Case(kind, [3, 4], 64, 256, 2)
    c.call()
    for name in ("a", "b", "sa", "sb", "offsets"):
        for value in (bad, None):
            keep = getattr(c, name)
            setattr(c, name, value)
            with pytest.raises(ValueError):
                c.call()
            setattr(c, name, keep)
    for kw in (dict(order=bad), dict(bias=bad), dict(out=bad), dict(top_k=0), dict(top_k=65), dict(order=c.order.long()),
               dict(out=torch.zeros(7, 63, device="cuda").bfloat16()), dict(offsets=None)):
        if "offsets" in kw:
            continue
        with pytest.raises(ValueError):
            c.call(**kw)
    for name, value in (("a", c.a[:, :-16]), ("b", c.b[:, :, :-16]), ("b", c.b[0]), ("sb", c.sb[:1]), ("sa", c.sa[:1]),
                        ("offsets", c.offsets[:-1]), ("offsets", c.offsets.long()), ("a", c.a.cpu()),
                        ("b", c.b.transpose(0, 1))):
        keep = getattr(c, name)
        setattr(c, name, value)
        with pytest.raises(ValueError):
            c.call()
        setattr(c, name, keep)
    c.order = None                                          # A has fewer rows than tokens' choices: other offsets
    assert c.call().shape[0] == c.m
