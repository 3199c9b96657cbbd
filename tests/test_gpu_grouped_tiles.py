"""GPU tests of the grouped GEMMs tile by tile, the tile that a call takes
asserted: sums that are exact in binary32, under scales of five powers of two,
by equality with the formula rounded once (one scale read from the wrong place
shows), and, on values of every size, the bits of the GEMM of the same name on
its tile of the same products."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

from tests.test_gpu_grouped import KINDS, Case, spread  # noqa: E402

PATH = {"i8": 0, "f8": 1, "mx8": 2, "mx4": 3, "block": 4}
WIDE, PANEL, STREAM, SMALL, SQUARE, TALL = 18, 17, 16, 8, 7, 5    # (blockscale's tall tile is 10)


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def tile_of(c):
    return q.select_grouped_tile(PATH[c.kind], c.rows, c.E, c.N)


# 17 to 90 rows an expert and the edges of the tiles' rows among them
MID = [20, 0, 90, 1, 64, 65, 77, 0, 17, 33, 96, 40, 0, 2, 100, 31]


def exact_case(kind, counts, N, K, top_k, extra):
    """Codes of small whole numbers (e2m1: halves up to 1.5) and scales 2^-2 to
    2^2: a product is a multiple of 2^-6 and at most 64, a sum of 2304 of them
    below 2^18, so every partial sum has at most 24 bits."""
    c = Case(kind, counts, N, K, top_k, extra=extra, seed=K + N)
    g = torch.Generator(device="cuda")
    g.manual_seed(K)

    def small(*s):
        return torch.randint(-2, 3, s, device="cuda", generator=g)
    if kind == "mx4":
        c.a, c.b = (torch.randint(0, 256, t.shape, device="cuda", generator=g, dtype=torch.uint8) & 0xbb
                    for t in (c.a, c.b))
    elif kind == "i8":
        c.a, c.b = small(*c.a.shape).to(torch.int8), small(*c.b.shape).to(torch.int8)
    else:
        c.a, c.b = (small(*t.shape).float().to(torch.float8_e4m3fn).view(torch.uint8) for t in (c.a, c.b))

    def power(t):
        e = torch.randint(-2, 3, t.shape, device="cuda", generator=g)
        return (e + 127).to(torch.uint8) if t.dtype == torch.uint8 else torch.exp2(e.float())
    c.sa, c.sb = power(c.sa), power(c.sb)
    c.bias = torch.randint(-8, 9, (c.E, N), device="cuda", generator=g).bfloat16()
    return c


def formula(c, e, at, n):
    rows = torch.arange(at, at + n, device="cuda")
    if c.order is not None:
        rows = c.order[rows].long() // c.top_k
    a, b = c._wide(c.a[rows], c.sa[rows], 1), c._wide(c.b[e], c.sb[e], 128 if c.kind == "block" else 1)
    if c.kind == "i8":
        a, b = a * c.sa[rows].double()[:, None], b * c.sb[e].double()[:, None]
    return (torch.mm(a, b.t().contiguous()) + c.bias[e].double()).bfloat16()


SHAPES = [(WIDE, MID, 3801, 384), (WIDE, MID, 3841, 1152), (WIDE, spread(3000, 50, 1), 2500, 640),
          (WIDE, spread(1500, 40, 2), 6000, 128), (WIDE, [23] * 64, 3330, 2304),
          (SQUARE, spread(1000, 16, 3), 641, 896), (PANEL, spread(200, 64, 4), 1041, 1152),
          (STREAM, spread(24, 12, 5), 1313, 896), (SMALL, spread(30, 40, 6), 40, 640),
          (TALL, spread(1200, 4, 7), 521, 1152)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tile,counts,N,K", SHAPES)
@pytest.mark.parametrize("top_k", [0, 3])
def test_exact_sums(kind, tile, counts, N, K, top_k):
    if kind == "block" and tile == TALL:
        tile, counts = 10, spread(5000, 4, 7)
    c = exact_case(kind, counts, N, K, top_k, extra=top_k)
    assert tile_of(c) == tile
    out = torch.full((c.rows, N + (-N) % 8), 9.0, dtype=torch.bfloat16, device="cuda")
    c.call(out=out[:, :N])
    at = 0
    for e, n in enumerate(counts):
        if n:
            assert torch.equal(out[at:at + n, :N], formula(c, e, at, n)), e
        at += n
    assert bool((out[at:] == 9).all()) and bool((out[:, N:] == 9).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("part", [0, 1, 2, -1])
def test_one_wrong_scale_shows(kind, part):
    """The other way round: the same comparison with one scale of the formula
    off by a factor of two fails in its row, or its columns."""
    c = exact_case(kind, MID, 3801, 384, 0, 0)
    out = c.call()
    e, at = 2, 20
    for name in ("sa", "sb"):
        keep = getattr(c, name)
        s = keep.clone()
        one = s[at + 7] if name == "sa" else s[e, 5]         # a row's scales, or a (block of) column's
        one = one if one.dim() == 0 else one[part % 3 if kind == "block" else part]
        one.copy_(one + 1 if s.dtype == torch.uint8 else one * 2)
        setattr(c, name, s)
        wrong = out[at:at + 90] != formula(c, e, at, 90)
        setattr(c, name, keep)
        if name == "sa":
            assert bool(wrong[7].any()) and not bool(wrong[:7].any()) and not bool(wrong[8:].any())
        else:
            cols = slice(5 * 128, 6 * 128) if kind == "block" else slice(5, 6)
            assert bool(wrong[:, cols].any())
            wrong[:, cols] = False
            assert not bool(wrong.any())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("tile,counts,N,K", [(WIDE, MID, 3801, 1152), (WIDE, spread(3000, 50, 8), 2500, 640),
                                             (WIDE, [40] * 32, 6200, 2048), (SQUARE, spread(1000, 16, 9), 641, 896),
                                             (TALL, [300, 5, 700, 256], 521, 1152)])
def test_same_bits_as_the_dense_gemm(kind, tile, counts, N, K):
    """On the tile of the same products: 128x128 for 128x256, 256x256 (of
    blockscale 256x128) for the tall one."""
    if kind == "block" and tile == TALL:
        tile, counts = 10, [2000, 5, 700, 256]
    c = Case(kind, counts, N, K, 2, bias=True, seed=N)
    assert tile_of(c) == tile
    out, at = c.call(), 0
    for e, n in enumerate(counts):
        if n == 0:
            continue
        rows = c.order[at:at + n].long() // 2
        args = (c.a[rows].contiguous(), c.b[e], c.sa[rows].contiguous(), c.sb[e].clone())
        q.force_tile(7 if tile == WIDE else tile)
        try:
            if kind.startswith("mx"):
                d = q.qgemm_mx(q.QGEMM_MX_E4M3 if kind == "mx8" else q.QGEMM_MX_E2M1, *args, 1, bias=c.bias[e])
            else:
                f = {"i8": q.qgemm_i8_rowwise, "f8": q.qgemm_f8_pertoken, "block": q.qgemm_f8_blockscale}[kind]
                d = f(*args, bias=c.bias[e])
        finally:
            q.force_tile(-1)
        assert torch.equal(d, out[at:at + n]), e
        at += n
