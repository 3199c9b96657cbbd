"""GPU tests of the 4-bit matvec by equality: x, weights and scales are small
whole numbers and powers of two, so that every sum is exact in binary32 in any
order and the result is the exact one rounded once to bf16."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

E2M1 = (0, .5, 1, 1.5, 2, 3, 4, 6, -0.0, -.5, -1, -1.5, -2, -3, -4, -6)


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def make(kind, M, N, K, group, seed, zeros=False, bias=False, srows=1):
    """|x| <= 8, |w - z| <= 15, e2m1 in halves, scales 1/2, 1 or 2: sums stay
    below 2^24 units of the smallest product up to K = 2^24 / (8 * 15 * 4)."""
    assert K * 8 * 15 * 4 < 1 << 24
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def ints(lo, hi, *shape, dtype=torch.float32):
        return torch.randint(lo, hi, shape, device="cuda", generator=g).to(dtype)
    d = {"x": ints(-8, 9, M, K).bfloat16(), "w": ints(0, 256, N, K // 2, dtype=torch.uint8), "zeros": None,
         "bias": ints(-99, 100, N).bfloat16() if bias else None}
    if kind == "mx":
        d["scales"] = ints(126, 129, -(-N // srows), K // 32, dtype=torch.uint8)
    else:
        d["scales"] = torch.exp2(ints(-1, 2, N, K // group)).bfloat16()
        if zeros:
            d["zeros"] = ints(0, 16, N, K // group, dtype=torch.uint8)
    return d


def want(kind, d, group, srows=1):
    x, N = d["x"].double(), d["w"].shape[0]
    K = x.shape[1]
    out = torch.empty(x.shape[0], N, dtype=torch.float64, device="cuda")
    table = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    for n in range(0, N, 8192):                     # in parts: the weights in 64 bits are 16 times their size
        w = d["w"][n:n + 8192]
        nib = torch.stack((w & 15, w >> 4), 2).view(-1, K // group, group)
        if kind == "mx":
            rows = torch.arange(n, min(n + 8192, N), device="cuda") // srows
            v = table[nib.int()] * torch.exp2(d["scales"][rows].double() - 127)[..., None]
        else:
            z = 8.0 if d["zeros"] is None else d["zeros"][n:n + 8192].double()[..., None]
            v = (nib.double() - z) * d["scales"][n:n + 8192].double()[..., None]
        out[:, n:n + 8192] = torch.matmul(x, v.view(-1, K).t())
    return out if d["bias"] is None else out + d["bias"].double()


def run(kind, d, srows=1):
    if kind == "mx":
        return q.qgemm_w4_matvec_mx(d["x"], d["w"], d["scales"], srows, bias=d["bias"])
    return q.qgemm_w4_matvec_i4(d["x"], d["w"], d["scales"], d["zeros"], bias=d["bias"])


def check(kind, d, group=32, srows=1):
    got, exact = run(kind, d, srows), want(kind, d, group, srows)
    assert exact.abs().max() < 1 << 22                  # in units of 1/4: exact in binary32
    assert torch.equal(got, exact.to(torch.bfloat16)), torch.nonzero(got != exact.to(torch.bfloat16))[:4]


@pytest.mark.parametrize("M", [9, 16])
@pytest.mark.parametrize("N,K", [(24576, 8192), (24577, 8192), (32768, 8192), (30000, 4224), (128256, 8192)])
def test_many_tiles_of_a_row_in_parts(M, N, K):
    """x of more than eight rows and K > 4096 goes in parts; the sums of 7 and
    more tiles a workgroup, kept between them, do not all find room in LDS."""
    check("mx", make("mx", M, N, K, 32, N + M))


@pytest.mark.parametrize("zeros", [False, True])
def test_many_tiles_of_a_row_in_parts_int4(zeros):
    check("i4", make("i4", 16, 32769, 8192, 32, 3, zeros), 32)


SHAPES = [(1, 50, 2048), (4, 50, 2048), (8, 50, 2048), (16, 50, 8192), (2, 40, 384), (17, 40, 384), (64, 8200, 384)]


def real(M, N, K, group, seed):
    d = make("i4", M, N, K, group, seed, True)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    d["x"] = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    return d


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("z", [0, 8, 15, None])
def test_weights_at_their_zero_point_add_nothing(M, N, K, group, z):
    d = real(M, N, K, group, M)
    if z is None:                                        # 8 where there are no zero points
        d["zeros"], z = None, 8
    else:
        d["zeros"][:7] = z
    d["w"][:7] = 17 * z
    d["x"][0] *= 2.0 ** 100
    out = run("i4", d)
    assert not bool(out[:, :7].any()) and bool((out[:, 7:] != 0).any())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_an_infinite_x(M, N, K, group):
    """Infinity times w - z: its sign, and NaN where they are equal; other rows
    keep their bits."""
    d = real(M, N, K, group, M)
    before = run("i4", d)
    row, k = M // 2, K - 3
    d["x"][row, k] = float("-inf")
    out = run("i4", d)
    diff = (d["w"][:, k // 2] >> 4 if k & 1 else d["w"][:, k // 2] & 15).float() - d["zeros"][:, k // group].float()
    exact = torch.where(diff == 0, float("nan"), diff * float("-inf"))
    assert torch.equal(out[row].isnan(), exact.isnan()) and torch.equal(out[row].nan_to_num(), exact.bfloat16().nan_to_num())
    keep = torch.arange(M, device="cuda") != row
    assert torch.equal(out[keep], before[keep])


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_sums_near_the_top_of_the_range(M, N, K, group):
    d = real(M, N, K, group, M)
    d["x"][:] = 2.0 ** 113
    d["w"][:] = 0x99
    d["zeros"][:] = 8
    d["scales"][:] = 1.0
    assert torch.equal(run("i4", d), torch.full((M, N), K * 2.0 ** 113, device="cuda").bfloat16())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_zero_points_of_eight_bits(M, N, K, group):
    d = make("i4", M, N, K, group, 7, True)
    d["zeros"] = torch.randint(0, 256, d["zeros"].shape, device="cuda", dtype=torch.uint8)
    d["x"] = d["x"].sign()
    check("i4", d, group)


@pytest.mark.parametrize("kind,group", [("i4", 32), ("i4", 128), ("mx", 32)])
@pytest.mark.parametrize("M", [1, 16])
def test_tables_that_are_not_16_byte_aligned(kind, group, M):
    d = make(kind, M, 200, 2048, group, 5, kind == "i4")
    for n in ("scales", "zeros"):
        if d[n] is not None:
            buf = torch.empty(d[n].numel() + 1, dtype=d[n].dtype, device="cuda")
            buf[1:] = d[n].view(-1)
            d[n] = buf[1:].view(d[n].shape)
            assert d[n].data_ptr() % 16
    check(kind, d, group)


# A workgroup that walks over several tiles of weights (256 or 512 workgroups of
# 16 rows each), whose last tile is not whole; K of 8, 57 and 64 chunks, the
# longest in parts above four rows.
@pytest.mark.parametrize("M", [1, 3, 4, 8, 16])
@pytest.mark.parametrize("N,K", [(8203, 1024), (12337, 7296), (20011, 8192)])
@pytest.mark.parametrize("kind,group,zeros,srows", [("i4", 32, True, 1), ("i4", 32, False, 1), ("i4", 64, True, 1),
                                                    ("i4", 64, False, 1), ("i4", 128, True, 1), ("i4", 128, False, 1),
                                                    ("mx", 32, False, 1), ("mx", 32, False, 32)])
def test_several_tiles_a_workgroup(kind, group, zeros, srows, M, N, K):
    check(kind, make(kind, M, N, K, group, M + N, zeros, True, srows), group, srows)


# Above 16 rows: one and two tiles of weights a wave, last tiles that are not
# whole, K that ends inside a chunk and K > 8192.
@pytest.mark.parametrize("M", [17, 32, 33, 64])
@pytest.mark.parametrize("N,K", [(8192, 1056), (8209, 8320), (530, 10240)])
@pytest.mark.parametrize("kind,group,zeros,srows", [("i4", 32, True, 1), ("i4", 64, False, 1), ("i4", 128, True, 1),
                                                    ("mx", 32, False, 1), ("mx", 32, False, 32)])
def test_many_rows(kind, group, zeros, srows, M, N, K):
    K = K // group * group
    check(kind, make(kind, M, N, K, group, M + N, zeros, True, srows), group, srows)


@pytest.mark.parametrize("M", [1, 4, 5, 16])
@pytest.mark.parametrize("K", [8320, 21504, 33024])
@pytest.mark.parametrize("kind,group,zeros", [("i4", 32, False), ("i4", 64, True), ("i4", 128, True), ("mx", 32, False)])
def test_long_rows(kind, group, zeros, M, K):
    check(kind, make(kind, M, 517, K, group, M + K, zeros, True), group)


@pytest.mark.parametrize("M,N,K", [(1, 12337, 5376), (16, 20011, 8192), (33, 8209, 2048), (1, 517, 21504)])
@pytest.mark.parametrize("kind", ["i4", "mx"])
def test_the_same_call_gives_the_same_bits(kind, M, N, K):
    d = make(kind, M, N, K, 32, 1, kind == "i4")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    d["x"] = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    first = run(kind, d)
    for _ in range(5):
        assert torch.equal(run(kind, d), first)
