"""GPU tests of the 8-bit cache with what is not a number: it comes out where
it went in, whatever kernel and number of splits the lengths lead to, and
nowhere else."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import block_scaled_precision_02_amd as q  # noqa: E402

from tests import kv8_ref  # noqa: E402
from tests.test_gpu_kv8 import Setup  # noqa: E402


@pytest.fixture(autouse=True)
def _gpu_only():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


HEADS, DIM = 8, 128


def splits(s, cache):
    need = q.lib().qgemm_kv8_attention_workspace(cache._ref, s.tokens, len(s.lens), HEADS, s.max_q, s.max_kv, 1, 0)
    return max(1, need // (s.tokens * HEADS * (DIM + 2) * 4))


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


# new tokens, cached tokens with them, the range of splits they lead to: one
# token unsplit, up to four splits, more; the same with 24 rows; many rows
SHAPES = [(1, 300, 1, 1), (1, 1500, 2, 4), (1, 9000, 5, 64), (3, 300, 1, 1), (3, 1500, 2, 4), (3, 9000, 5, 64),
          (50, 300, 1, 1), (50, 3000, 5, 64)]


@pytest.mark.parametrize("n_q,n,least,most", SHAPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_row(n_q, n, least, most, bad):
    s = Setup("e4m3", 1, DIM, 64, [(n_q, n)], seed=n)
    cache, Q = s.gpu(), s.bf16(s.tokens, HEADS, DIM).cuda()
    assert least <= splits(s, cache) <= most
    args = s.seqs() + (s.max_q, s.max_kv)
    want = q.qgemm_kv8_attention(cache, Q, *args)
    t = n_q // 2
    Q[t, 5, 77] = bad
    got = q.qgemm_kv8_attention(cache, Q, *args)
    assert bool(got[t, 5].isnan().all())
    got[t, 5] = want[t, 5]
    assert same(got, want)


def test_query_rows_that_see_nothing():
    for n_q, n in ((4, 3), (60, 3)):
        s = Setup("e4m3", 1, DIM, 64, [(n_q, n)], seed=n_q)
        Q = s.bf16(s.tokens, HEADS, DIM).cuda()
        Q[:n_q - n] = float("nan")
        out = q.qgemm_kv8_attention(s.gpu(), Q, *s.seqs(), s.max_q, s.max_kv)
        assert not bool(out[:n_q - n].any()) and bool(out[n_q - n:].isfinite().all())


@pytest.mark.parametrize("exponent", [-126, -101, -100, -81, -60, 115, 120])
@pytest.mark.parametrize("n_q,n", [(1, 700), (1, 20000), (50, 20000)])
def test_v_scales_at_the_ends(exponent, n_q, n):
    """All keys alike and every V scale tiny (or huge): the sums stay in
    range; scales below 2^-100 are read as 2^-100."""
    s = Setup("i8", 1, DIM, 64, [(n_q, n)], seed=n)
    s.cache["k_scale"].zero_()
    if exponent == 120:
        s.cache["v"].bitwise_and_(63)                   # results within bf16
    s.cache["v_scale"].fill_(2.0 ** exponent)
    Q = s.bf16(s.tokens, HEADS, DIM)
    out = q.qgemm_kv8_attention(s.gpu(), Q.cuda(), *s.seqs(), s.max_q, s.max_kv).float().cpu()
    s.cache["v_scale"].fill_(2.0 ** max(exponent, -100))
    want, tol = kv8_ref.attention(s.cache, Q, s.table.tolist(), s.cu, s.lens, "i8")
    assert (np.abs(out.double().numpy() - want) <= tol).all()


BAD = [float("nan"), float("inf"), float("-inf")]
NAMES = ("k", "v", "k_scale", "v_scale")


def held(cache):
    return {n: getattr(cache, n).view(torch.uint8).clone() for n in NAMES}


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", BAD)
@pytest.mark.parametrize("seqs", [[(1, 70), (1, 9)], [(90, 150), (3, 20)]])
def test_append_shows_it_in_the_scale(fmt, which, bad, seqs):
    s = Setup(fmt, 3, 64, 32, seqs, seed=4)
    new = {n: s.bf16(s.tokens, 3, 64).cuda() for n in "kv"}
    table, cu, lens = s.seqs()
    good, cache = s.gpu(), s.gpu()
    q.qgemm_kv8_append(good, new["k"], new["v"], table, cu, lens, s.max_q)
    new[which][s.cu[1] - 1, 1, 33] = bad                    # the first sequence's last token, head 1
    q.qgemm_kv8_append(cache, new["k"], new["v"], table, cu, lens, s.max_q)
    n = s.lens[0]
    blk = s.table[0, (n - 1) // 32]
    name = which + "_scale"
    assert bool(getattr(cache, name)[blk, 1].isnan()) and bool(getattr(good, name)[blk, 1].isfinite())
    a, b = held(cache), held(good)
    hit = getattr(cache, which)[blk, 1].view(torch.uint8)
    past = hit[n % 32:] if which == "k" else hit[:, n % 32:]
    was = getattr(good, which)[blk, 1].view(torch.uint8)
    assert torch.equal(past, was[n % 32:] if which == "k" else was[:, n % 32:])
    for d in (a, b):                                        # everything else keeps its bits
        d[which][blk, 1] = 0
        d[name].view(torch.float32)[blk, 1] = 0
    for x in NAMES:
        assert torch.equal(a[x], b[x]), x
    # a finite token more: the scale stays; the block begun anew: it is gone
    one = torch.ones(1, 3, 64, device="cuda").bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q.qgemm_kv8_append(cache, one, one, table[:1], i32(0, 1), i32(n + 1), 1)
    assert bool(getattr(cache, name)[blk, 1].isnan())
    q.qgemm_kv8_append(cache, one, one, table[:1], i32(0, 1), i32((n - 1) // 32 * 32 + 1), 1)
    assert bool(getattr(cache, name)[blk, 1].isfinite())


@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("n_q,n,window", [(1, 300, 0), (1, 1500, 0), (1, 9000, 0), (6, 300, 40), (3, 9000, 0),
                                          (200, 500, 0), (200, 500, 70), (50, 3000, 0), (300, 300, 0)])
def test_rows_that_see_a_block_without_a_scale(which, fmt, n_q, n, window):
    s = Setup(fmt, 2, DIM, 32, [(n_q, n), (2, 100)], seed=n)
    s.cache["v_scale"][s.table[0, 2::3], 1] = 0.0            # blocks whose scale is zero, beside and behind it
    j = max(0, n - n_q // 2 - 20) // 32
    s.cache["v_scale"][s.table[0, j], 1] = 0.01
    Q = s.bf16(s.tokens, HEADS, DIM).cuda()
    args = s.seqs() + (s.max_q, s.max_kv)
    want = q.qgemm_kv8_attention(s.gpu(), Q, *args, window=window)
    s.cache[which][s.table[0, j], 1] = float("nan")
    got = q.qgemm_kv8_attention(s.gpu(), Q, *args, window=window)
    at = n - n_q + torch.arange(n_q, device="cuda")          # positions of the first sequence's new tokens
    sees = at >= 32 * j
    if window:
        sees &= at - window < 32 * j + 31
    rows = torch.nonzero(sees).flatten()
    assert len(rows) and bool(got[rows, HEADS // 2:].isnan().all())
    got[rows, HEADS // 2:] = want[rows, HEADS // 2:]
    assert same(got, want)
