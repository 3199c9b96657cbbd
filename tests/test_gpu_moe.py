"""GPU tests of the sort by experts and of the rows' way to the experts and
back: the sort against lists in numpy, the copies by equality, sums and
gradients against 64 bits within the roundings they have, against differences
and one another; choices without expert, odd sizes, strides, other streams, a
replayed graph, nothing outside the outputs written."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def routed(tokens, k, experts, seed, total=None):
    """ids int32 [tokens, k], k different ones of total experts (those past
    `experts` or below 0 another rank's), some chosen more often."""
    rng = np.random.default_rng(seed)
    total = total or experts
    if k <= total and tokens * total <= 1 << 22:
        key = rng.random((tokens, total)) ** (1.0 + 3.0 * rng.random(total))
        ids = np.argsort(key, 1)[:, :k]
    else:
        ids = rng.integers(0, total, (tokens, k))
    return torch.from_numpy((ids - (total - experts) // 2).astype(np.int32)).cuda()


def lists(ids, experts):
    """(offsets, order, position) from the definition."""
    flat = ids.cpu().numpy().reshape(-1)
    order = np.full(flat.size, -1, np.int32)
    position = np.full(flat.size, -1, np.int32)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    by = np.argsort(key, kind="stable")
    offsets = np.searchsorted(key[by], np.arange(experts + 1)).astype(np.int32)
    n = offsets[-1]
    order[:n] = by[:n]
    position[by[:n]] = np.arange(n)
    return offsets, order, position.reshape(ids.shape)


def check_sort(ids, experts, got):
    for a, b in zip(got, lists(ids, experts)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("tokens,k,experts", [(1, 1, 1), (1, 8, 256), (3, 2, 5), (64, 8, 256), (63, 6, 64), (1000, 8, 1024),
                                              (1024, 8, 128), (1025, 8, 128), (2731, 3, 7), (9000, 1, 2), (16385, 8, 256),
                                              (40000, 8, 129), (524289, 2, 1000)])
def test_sort(tokens, k, experts):
    ids = routed(tokens, k, experts, tokens + k)
    check_sort(ids, experts, q.qgemm_moe_sort(ids, experts))


@pytest.mark.parametrize("tokens,k,experts,total", [(5, 4, 8, 32), (100, 8, 32, 256), (3000, 8, 16, 128)])
def test_sort_of_one_rank(tokens, k, experts, total):
    ids = routed(tokens, k, experts, 7, total)
    assert bool(((ids < 0) | (ids >= experts)).any())
    check_sort(ids, experts, q.qgemm_moe_sort(ids, experts))


@pytest.mark.parametrize("tokens", [7, 3001])
def test_sort_of_uneven_choices(tokens):
    for ids in (torch.full((tokens, 3), 4), torch.full((tokens, 3), -1), torch.full((tokens, 3), 9),
                torch.full((tokens, 3), -2 ** 31), torch.full((tokens, 3), 2 ** 31 - 1),
                torch.arange(tokens * 3).view(tokens, 3) % 2 * 8):
        ids = ids.int().cuda()
        check_sort(ids, 9, q.qgemm_moe_sort(ids, 9))


def test_sort_of_nothing():
    offsets, order, position = q.qgemm_moe_sort(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 300)
    assert offsets.tolist() == [0] * 301 and order.numel() == 0 and tuple(position.shape) == (0, 4)


@pytest.mark.parametrize("tokens", [50, 5000])
def test_sort_into_given_memory_and_graph(tokens):
    k, E = 4, 40
    ids = routed(tokens, k, E, 3)
    slots = tokens * k
    bufs = [torch.full((n + 8,), 77, dtype=torch.int32, device="cuda") for n in (E + 1, slots, slots)]
    outs = [b[:n] for b, n in zip(bufs, (E + 1, slots, slots))]
    need = q.lib().qgemm_moe_sort_workspace(tokens, k, E)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    kw = dict(offsets=outs[0], order=outs[1], position=outs[2].view(tokens, k), workspace=ws)
    check_sort(ids, E, q.qgemm_moe_sort(ids, E, **kw))
    assert all(bool((b[n:] == 77).all()) for b, n in zip(bufs, (E + 1, slots, slots)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qgemm_moe_sort(ids, E, **kw)
    for seed in range(3):
        ids.copy_(routed(tokens, k, E, 10 + seed, 2 * E))
        graph.replay()
        torch.cuda.synchronize()
        check_sort(ids, E, outs[:2] + [outs[2].view(tokens, k)])


# ------------------------------------------------------------ exchange

def data(tokens, k, experts, H, seed, total=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    ids = routed(tokens, k, experts, seed, total)
    offsets, order, position = q.qgemm_moe_sort(ids, experts)

    def bf16(*s):
        return torch.randn(*s, device="cuda", generator=g).bfloat16()
    w = torch.rand(tokens, k, device="cuda", generator=g)
    return position, w, bf16(tokens, H), bf16(tokens * k, H), bf16(tokens, H)


def dense(position, rows):
    """float64 [tokens, k, rows] of ones where a choice has a row."""
    p = position.long()
    m = torch.zeros(*p.shape, rows, dtype=torch.float64, device="cuda")
    t, j = torch.nonzero(p >= 0, as_tuple=True)
    m[t, j, p[t, j]] = 1
    return m


SIZES = [(1, 1, 8), (1, 8, 7168), (5, 3, 1032), (64, 8, 2048), (33, 64, 264), (130, 6, 5376), (7, 2, 16384 + 2056)]


@pytest.mark.parametrize("tokens,k,H", SIZES)
@pytest.mark.parametrize("total", [64, 200])
def test_gather(tokens, k, H, total):
    position, w, x, y, r = data(tokens, k, 64, H, tokens, total)
    base = y.clone()
    out = q.qgemm_moe_gather(x, position, out=y)
    assert out is y
    p = position.view(-1).long()
    live = p >= 0
    base[p[live]] = x.repeat_interleave(k, 0)[live]
    assert torch.equal(y.view(torch.int16), base.view(torch.int16))


def half(t):
    """Half a step of bf16, and a little for the end of the range."""
    return t.abs() * 2.0 ** -8 + 2.0 ** -134


@pytest.mark.parametrize("tokens,k,H", SIZES)
@pytest.mark.parametrize("total", [64, 200])
def test_combine(tokens, k, H, total):
    position, w, x, y, r = data(tokens, k, 64, H, tokens, total)
    m = dense(position, tokens * k)
    for weights in (w, None):
        for residual in (r, None):
            got = q.qgemm_moe_combine(y, position, weights, residual=residual).double()
            mw = (m * (w.double()[..., None] if weights is not None else 1)).sum(1)
            want, size = mw @ y.double(), mw @ y.double().abs()
            if residual is not None:
                want, size = want + r.double(), size + r.double().abs()
            # k + 1 binary32 roundings of terms no larger than the sum of magnitudes
            assert bool(((got - want).abs() <= half(want) + 1.01 * (k + 1) * 2.0 ** -24 * size).all())


@pytest.mark.parametrize("tokens,k,H", SIZES)
@pytest.mark.parametrize("total", [64, 200])
def test_gradient(tokens, k, H, total):
    position, w, x, y, dout = data(tokens, k, 64, H, tokens, total)
    dY = torch.full_like(y, 3.0)
    got, dw = q.qgemm_moe_combine_grad(dout, y, position, w, dY=dY)
    assert got is dY
    m = dense(position, tokens * k)
    mw = (m * w.double()[..., None]).sum(1)
    want = mw.t() @ dout.double()
    taken = (m.sum((0, 1)) > 0)[:, None]
    assert bool((torch.where(taken, want, 3.0) - got.double()).abs().le(
        torch.where(taken, half(want) + want.abs() * 2.0 ** -23, 0.0)).all())
    p = position.clamp(min=0).long()
    prod = dout.double()[:, None, :] * y.double()[p]
    live = position >= 0
    # a binary32 sum of H exact products, in any order
    err = (dw.double() - torch.where(live, prod.sum(2), 0.0)).abs()
    assert bool((err <= H * 2.0 ** -24 * torch.where(live, prod.abs().sum(2), 0.0)).all())
    # in place, and the same bits again
    mine = y.clone()
    again, dw2 = q.qgemm_moe_combine_grad(dout, mine, position, w, dY=mine)
    assert torch.equal(torch.where(taken, again, 0), torch.where(taken, got, 0)) and torch.equal(dw, dw2)
    # the gather's gradient: the sum over a token's rows
    dx = q.qgemm_moe_combine(y, position).double()
    want = m.sum(1) @ y.double()
    assert bool(((dx - want).abs() <= half(want) + 1.01 * k * 2.0 ** -24 * (m.sum(1) @ y.double().abs())).all())


def test_gradient_against_differences():
    """<dout, combine> moves by its gradients' products with the step.  Values
    on a coarse grid, so that every sum is exact in bf16 and binary32."""
    position, w, x, y, r = data(6, 3, 8, 64, 1, 12)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)

    def grid(*s):
        return torch.randint(-2, 3, s, device="cuda", generator=g).float()
    y, dy, dout = grid(18, 64).bfloat16(), grid(18, 64).bfloat16(), grid(6, 64).bfloat16()
    w, dw = grid(6, 3), grid(6, 3)

    def loss(y, w):
        return (q.qgemm_moe_combine(y, position, w).double() * dout.double()).sum().item()
    gy, gw = q.qgemm_moe_combine_grad(dout, y, position, w, dY=torch.zeros_like(y))
    assert loss((y + dy).bfloat16(), w) - loss(y, w) == (gy.double() * dy.double()).sum().item()
    assert loss(y, w + dw) - loss(y, w) == (gw.double() * dw.double()).sum().item()


def test_what_is_not_finite_stays_in_its_rows():
    position, w, x, y, r = data(20, 4, 8, 256, 2, 16)
    free = torch.ones(80, dtype=torch.bool, device="cuda")
    free[position[position >= 0].long()] = False
    assert bool(free.any())
    y[free] = float("nan")                               # rows that no slot has
    w[position < 0] = float("nan")                       # weights of choices without expert
    assert bool(q.qgemm_moe_combine(y, position, w, residual=r).isfinite().all())
    dY, dw = q.qgemm_moe_combine_grad(r, y, position, w, dY=torch.zeros_like(y))
    assert bool(dY.isfinite().all()) and bool(dw.isfinite().all())
    t, j = [int(v[0]) for v in torch.nonzero(position >= 0, as_tuple=True)]
    y[position[t, j], 17] = float("inf")
    out = q.qgemm_moe_combine(y, position, w, residual=r)
    bad = ~out.isfinite()
    assert bool(bad[t, 17]) and int(bad.sum()) == 1


def test_strides_and_rows_that_are_not_there():
    tokens, k, H = 9, 3, 520
    position, w, x, y, r = data(tokens, k, 16, H, 3)
    want = q.qgemm_moe_combine(y, position, w, residual=r)
    xs = q.qgemm_moe_gather(x, position)
    dY, dw = q.qgemm_moe_combine_grad(r, y, position, w)

    def wide(t, fill=9.0):
        b = torch.full((t.shape[0] + 1, H + 24), fill, dtype=torch.bfloat16, device="cuda")
        v = b[:t.shape[0], 8:8 + H]
        v.copy_(t)
        return b, v

    def kept(b):
        return bool((b[-1] == 9).all()) and bool((b[:, :8] == 9).all()) and bool((b[:, 8 + H:] == 9).all())
    (_, yv), (_, rv), (_, xv), (ob, ov), (gb, gv), (db, dv) = map(wide, (y, r, x, want, xs, dY))
    ov.zero_(), gv.zero_(), dv.zero_()
    assert torch.equal(q.qgemm_moe_combine(yv, position, w, residual=rv, out=ov), want) and kept(ob)
    assert torch.equal(q.qgemm_moe_gather(xv, position, out=gv), xs) and kept(gb)
    dw2 = q.qgemm_moe_combine_grad(rv, yv, position, w, dY=dv)[1]
    assert torch.equal(dv, dY) and torch.equal(dw2, dw) and kept(db)
    # fewer rows than the positions name: those past the end are no experts
    n = tokens * k // 2
    some = torch.where(position < n, position, -1)
    for a, b in ((q.qgemm_moe_combine(y[:n], position, w), q.qgemm_moe_combine(y, some, w)),
                 (q.qgemm_moe_combine(y[:0], position, w, residual=r), r)):
        assert torch.equal(a, b)
    few = torch.zeros(n, H, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(q.qgemm_moe_gather(x, position, out=few), xs[:n])
    odd = torch.where(position == 0, -2 ** 31, torch.where(position == 1, 2 ** 31 - 1, position))
    assert torch.equal(q.qgemm_moe_combine(y, odd, w),
                       q.qgemm_moe_combine(y, torch.where(position < 2, -1, position), w))
    own = r.clone()
    assert torch.equal(q.qgemm_moe_combine(y, position, w, residual=own, out=own), want)


def test_empty_calls():
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    row = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    assert q.qgemm_moe_gather(row, none).shape == (0, 64)
    assert q.qgemm_moe_combine(row, none).shape == (0, 64)
    dY, dw = q.qgemm_moe_combine_grad(row, row, none, torch.zeros(0, 4, device="cuda"))
    assert dY.shape == (0, 64) and dw.shape == (0, 4)


def test_streams_and_graph():
    tokens, k, H = 70, 4, 1024
    position, w, x, y, r = data(tokens, k, 16, H, 4)
    want = (q.qgemm_moe_gather(x, position), q.qgemm_moe_combine(y, position, w, residual=r),
            *q.qgemm_moe_combine_grad(r, y, position, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (q.qgemm_moe_gather(x, position, stream=side), q.qgemm_moe_combine(y, position, w, residual=r, stream=side),
           *q.qgemm_moe_combine_grad(r, y, position, w, stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    outs = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.qgemm_moe_gather(x, position, out=outs[0])
        q.qgemm_moe_combine(y, position, w, residual=r, out=outs[1])
        q.qgemm_moe_combine_grad(r, y, position, w, dY=outs[2], dweights=outs[3])
    for _ in range(3):
        x.mul_(0.5), y.mul_(0.75), w.mul_(1.5)
        want = (q.qgemm_moe_gather(x, position), q.qgemm_moe_combine(y, position, w, residual=r),
                *q.qgemm_moe_combine_grad(r, y, position, w))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


@pytest.mark.parametrize("bad", [7, [1.0], "x", None])
def test_refusals(bad):
    position, w, x, y, r = data(4, 2, 8, 64, 5)
    ids = position.clone()
    for call in (lambda: q.qgemm_moe_sort(bad, 8), lambda: q.qgemm_moe_sort(ids.long(), 8),
                 lambda: q.qgemm_moe_sort(ids, 0), lambda: q.qgemm_moe_sort(ids, 1025),
                 lambda: q.qgemm_moe_sort(ids, 2.0), lambda: q.qgemm_moe_sort(ids.view(-1), 8),
                 lambda: q.qgemm_moe_sort(ids.t(), 8), lambda: q.qgemm_moe_sort(ids.cpu(), 8),
                 lambda: q.qgemm_moe_sort(ids, 8, offsets=ids), lambda: q.qgemm_moe_sort(ids, 8, workspace=4),
                 lambda: q.qgemm_moe_gather(bad, position), lambda: q.qgemm_moe_gather(x, bad),
                 lambda: q.qgemm_moe_gather(x[:3], position), lambda: q.qgemm_moe_gather(x.float(), position),
                 lambda: q.qgemm_moe_gather(x, position, out=y[:, :32]),
                 lambda: q.qgemm_moe_gather(x[:, :60], position),
                 lambda: q.qgemm_moe_combine(bad, position), lambda: q.qgemm_moe_combine(y, bad),
                 lambda: q.qgemm_moe_combine(y, position, w.double()), lambda: q.qgemm_moe_combine(y, position, w[:2]),
                 lambda: q.qgemm_moe_combine(y, position, w, residual=r[:2]),
                 lambda: q.qgemm_moe_combine(y, position, w, out=y),
                 lambda: q.qgemm_moe_combine_grad(bad, y, position, w),
                 lambda: q.qgemm_moe_combine_grad(r, bad, position, w),
                 lambda: q.qgemm_moe_combine_grad(r, y, position, bad),
                 lambda: q.qgemm_moe_combine_grad(r, y, position, w, dY=r),
                 lambda: q.qgemm_moe_combine_grad(r, y, position, w, dweights=w.double())):
        with pytest.raises(ValueError):
            call()
