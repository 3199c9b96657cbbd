"""The decoder-layer entry points on the CPU: bad arguments are refused with
the documented status before any HIP call (fake device pointers that nothing
dereferences), empty calls are no-ops, a wrong device is named."""
import pytest

import block_scaled_precision_02_amd as q

A, B, C, D, E = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000


def norm(name="f8_pertoken", fmt=0, X=A, ldx=128, R=B, ldr=128, gamma=C, eps=1e-6, Rout=B, ldo=128, Q=D, ldq=128, S=E,
         lds=4, M=2, K=128):
    f = getattr(q.lib(), "qgemm_rmsnorm_quant_" + name)
    head = (fmt,) if name == "mx" else ()
    tail = (lds,) if name in ("mx", "f8_block") else ()
    return f(*head, X, ldx, R, ldr, gamma, eps, Rout, ldo, Q, ldq, S, *tail, M, K, None)


NORMS = ["i8_rowwise", "f8_pertoken", "f8_block", "mx"]


@pytest.mark.parametrize("name", NORMS)
@pytest.mark.parametrize("kw,status", [
    (dict(X=None), q.QGEMM_ERR_NULL_POINTER), (dict(gamma=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(Q=None), q.QGEMM_ERR_NULL_POINTER), (dict(S=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(M=-1), q.QGEMM_ERR_BAD_SHAPE), (dict(K=0), q.QGEMM_ERR_BAD_SHAPE), (dict(K=120), q.QGEMM_ERR_BAD_SHAPE),
    (dict(M=1 << 31), q.QGEMM_ERR_BAD_SHAPE), (dict(K=1 << 31), q.QGEMM_ERR_BAD_SHAPE),
    (dict(eps=-1.0), q.QGEMM_ERR_BAD_SHAPE), (dict(eps=float("nan")), q.QGEMM_ERR_BAD_SHAPE),
    (dict(X=A + 8), q.QGEMM_ERR_BAD_LAYOUT), (dict(R=B + 2), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(Rout=B + 2), q.QGEMM_ERR_BAD_LAYOUT), (dict(gamma=C + 4), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(Q=D + 8), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldx=120), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(ldx=132), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldr=64), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(ldo=129), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldq=120), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(ldq=136), q.QGEMM_ERR_BAD_LAYOUT),
])
def test_norm_refusals(name, kw, status):
    assert norm(name, **kw) == status
    assert q.lib().qgemm_last_error()


def test_norm_refusals_by_kind():
    assert norm("f8_block", K=96, ldx=96, ldr=96, ldo=96) == q.QGEMM_ERR_BAD_SHAPE
    assert norm("f8_block", lds=0) == q.QGEMM_ERR_BAD_LAYOUT
    assert norm("mx", lds=3) == q.QGEMM_ERR_BAD_LAYOUT
    assert norm("mx", fmt=2) == q.QGEMM_ERR_BAD_FORMAT
    assert norm("f8_pertoken", S=E + 2) == q.QGEMM_ERR_BAD_LAYOUT


@pytest.mark.parametrize("name", NORMS)
def test_norm_empty_and_device(name, monkeypatch):
    assert norm(name, M=0, X=None, R=None, gamma=None, Rout=None, Q=None, S=None) == q.QGEMM_OK
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx1201")
    assert norm(name) == q.QGEMM_ERR_UNSUPPORTED_DEVICE
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setenv("QGEMM_INJECT_LAUNCH_ERROR", "719")
    assert norm(name) == q.QGEMM_ERR_HIP
    assert b"injected" in q.lib().qgemm_last_error()
