"""GPU tests of the cache attention at the limits that a call names: tokens past
max_q are not computed, keys at and past max_kv not seen."""
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


@pytest.mark.parametrize("n_q,n,max_kv,window", [(1, 300, 200, 0), (1, 300, 195, 150), (1, 9000, 8001, 0), (3, 2000, 1201, 1999),
                                                 (70, 500, 333, 0), (70, 500, 470, 100), (50, 3000, 2500, 0)])
def test_keys_past_max_kv_are_not_seen(n_q, n, max_kv, window):
    s = Setup("e4m3", 1, 128, 64, [(n_q, n), (1, 60)], seed=n)
    Q = s.bf16(s.tokens, 8, 128)
    out = q.qgemm_kv8_attention(s.gpu(), Q.cuda(), *s.seqs(), s.max_q, max_kv, window=window)
    want, tol = reference(s, Q, max_kv, window)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


def reference(s, Q, max_kv, window):
    """kv8_ref.attention with the keys from max_kv on hidden: rows that see some
    of them are taken alone, as single tokens of a sequence that ends before."""
    cache, table = s.cache, s.table.tolist()
    want, tol = kv8_ref.attention(cache, Q, table, s.cu, s.lens, s.fmt, True, window)
    for b, n in enumerate(s.lens):
        nq = s.cu[b + 1] - s.cu[b]
        for t in range(nq):
            at = n - nq + t
            if at < max_kv:
                continue
            row, lo = s.cu[b] + t, max(0, at + 1 - window) if window else 0
            if lo >= max_kv:
                want[row], tol[row] = 0, 0
                continue
            w = max_kv - lo if window else 0
            want[row:row + 1], tol[row:row + 1] = kv8_ref.attention(cache, Q[row:row + 1], [table[b]], [0, 1], [max_kv],
                                                                    s.fmt, True, w)
    return want, tol


@pytest.mark.parametrize("n_q,max_q,n", [(5, 2, 100), (6, 3, 300), (6, 3, 5000), (90, 61, 300), (90, 61, 4000)])
def test_tokens_past_max_q_are_not_computed(n_q, max_q, n):
    s = Setup("e4m3", 1, 128, 64, [(n_q, n), (1, 60)], seed=n)
    Q = s.bf16(s.tokens, 8, 128).cuda()
    args = s.seqs()
    want = q.qgemm_kv8_attention(s.gpu(), Q, *args, s.max_q, s.max_kv)
    out = torch.full_like(want, 7.0)
    q.qgemm_kv8_attention(s.gpu(), Q, *args, max_q, s.max_kv, out=out)
    assert bool((out[max_q:n_q] == 7.0).all())
    keep = [t for t in range(s.tokens) if not max_q <= t < n_q]
    assert (out[keep].float() - want[keep].float()).abs().max() <= 2.0 ** -7 * want.abs().max()
