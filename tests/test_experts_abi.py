"""The entry points of a layer of experts, and the norm after a block, on the
CPU: bad arguments are refused with the documented status before any HIP call
(fake device pointers that nothing dereferences), empty calls are no-ops, a
wrong device is named."""
import ctypes as c

import pytest

import block_scaled_precision_02_amd as q


class Postnorm(c.Structure):
    _fields_ = [(n, c.c_void_p) for n in ("Y", "R", "gamma_post", "gate", "gamma", "Rout")] + \
        [(n, c.c_int64) for n in ("ldy", "ldr", "ldo")] + [("eps", c.c_float), ("alpha", c.c_float)]

A, B, C, D, E, F = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000
NULL, SHAPE, LAYOUT, FORMAT = (q.QGEMM_ERR_NULL_POINTER, q.QGEMM_ERR_BAD_SHAPE, q.QGEMM_ERR_BAD_LAYOUT,
                               q.QGEMM_ERR_BAD_FORMAT)


def sort(ids=A, tokens=4, top_k=2, experts=8, offsets=B, order=C, position=D, ws=None, nbytes=0):
    return q.lib().qgemm_moe_sort(ids, tokens, top_k, experts, offsets, order, position, ws, nbytes, None)


def gather(X=A, ldx=64, position=B, Y=C, ldy=64, tokens=4, top_k=2, rows=8, H=64):
    return q.lib().qgemm_moe_gather(X, ldx, position, Y, ldy, tokens, top_k, rows, H, None)


def combine(Y=A, ldy=64, position=B, weights=C, R=D, ldr=64, O=E, ldo=64, tokens=4, top_k=2, rows=8, H=64):
    return q.lib().qgemm_moe_combine(Y, ldy, position, weights, R, ldr, O, ldo, tokens, top_k, rows, H, None)


def grad(dO=A, lddo=64, Y=B, ldy=64, position=C, weights=D, dY=E, lddy=64, dw=F, tokens=4, top_k=2, rows=8, H=64):
    return q.lib().qgemm_moe_combine_grad(dO, lddo, Y, ldy, position, weights, dY, lddy, dw, tokens, top_k, rows, H, None)


def swiglu(name="f8_pertoken", fmt=0, X=A, ldx=256, count=None, Q=B, ldq=128, S=C, lds=4, M=2, I=128):
    f = getattr(q.lib(), "qgemm_swiglu_quant_" + name)
    head = (fmt,) if name == "mx" else ()
    tail = (lds,) if name in ("mx", "f8_block") else ()
    return f(*head, X, ldx, count, Q, ldq, S, *tail, M, I, None)


def postnorm(name="f8_pertoken", fmt=0, Q=F, ldq=128, S=A, lds=4, M=2, K=128, norm="ok", **kw):
    d = dict(Y=A, R=B, gamma_post=C, gate=D, gamma=E, Rout=B, ldy=128, ldr=128, ldo=128, eps=1e-6, alpha=1.0)
    d.update(kw)
    f = getattr(q.lib(), "qgemm_postnorm_quant_" + name)
    s = Postnorm(**d)
    head = (fmt,) if name == "mx" else ()
    tail = (lds,) if name in ("mx", "f8_block") else ()
    return f(*head, c.addressof(s) if norm == "ok" else norm, Q, ldq, S, *tail, M, K, None)


def grouped(name="i8_rowwise", fmt=0, A=A, lda=256, a_rows=4, B=B, ldb=256, sa=C, sb=D, offsets=E, order=F, top_k=2,
            bias=None, C_=A, ldc=64, rows=8, experts=3, N=64, K=256):
    f = getattr(q.lib(), f"qgemm_{name}_grouped")
    head = (fmt,) if name == "mx" else ()
    return f(*head, A, lda, a_rows, B, ldb, sa, sb, offsets, order, top_k, bias, C_, ldc, rows, experts, N, K, None)


CHOICES = [(dict(tokens=-1), SHAPE), (dict(top_k=0), SHAPE), (dict(top_k=65), SHAPE), (dict(tokens=1 << 30), SHAPE),
           (dict(tokens=1 << 29), SHAPE)]


@pytest.mark.parametrize("kw,status", CHOICES + [
    (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE), (dict(ids=None), NULL), (dict(offsets=None), NULL),
    (dict(order=None), NULL), (dict(position=None), NULL), (dict(ids=A + 2), LAYOUT), (dict(offsets=B + 1), LAYOUT),
    (dict(order=C + 2), LAYOUT), (dict(position=D + 2), LAYOUT), (dict(tokens=100000), NULL),
    (dict(tokens=100000, ws=E, nbytes=10), LAYOUT), (dict(tokens=100000, ws=E + 4, nbytes=1 << 30), LAYOUT)])
def test_sort_refusals(kw, status):
    assert sort(**kw) == status
    assert q.lib().qgemm_last_error()


def test_sort_workspace():
    size = q.lib().qgemm_moe_sort_workspace
    assert size(0, 8, 64) == 0 and size(64, 8, 256) == 0
    assert size(100000, 8, 64) > 0 and size(100000, 8, 64) % (64 * 4) == 0
    assert size(-1, 8, 64) == size(4, 0, 64) == size(4, 2, 0) == size(1 << 30, 1, 4) == -1
    assert size((1 << 30) - 1, 1, 1024) == 256 * 1024 * 4


ROWS = [(dict(rows=-1), SHAPE), (dict(rows=1 << 31), SHAPE), (dict(H=0), SHAPE), (dict(H=60), SHAPE),
        (dict(position=None), NULL), (dict(position=A + 2), LAYOUT)]


@pytest.mark.parametrize("kw,status", CHOICES + ROWS + [
    (dict(X=None), NULL), (dict(Y=None), NULL), (dict(X=A + 8), LAYOUT), (dict(Y=A + 2), LAYOUT),
    (dict(ldx=56), LAYOUT), (dict(ldx=68), LAYOUT), (dict(ldy=56), LAYOUT)])
def test_gather_refusals(kw, status):
    assert gather(**kw) == status


@pytest.mark.parametrize("kw,status", CHOICES + ROWS + [
    (dict(Y=None), NULL), (dict(O=None), NULL), (dict(Y=A + 8), LAYOUT), (dict(R=A + 2), LAYOUT),
    (dict(O=A + 2), LAYOUT), (dict(weights=A + 2), LAYOUT), (dict(ldy=56), LAYOUT), (dict(ldr=68), LAYOUT),
    (dict(ldo=56), LAYOUT)])
def test_combine_refusals(kw, status):
    assert combine(**kw) == status


@pytest.mark.parametrize("kw,status", CHOICES + ROWS + [
    (dict(dO=None), NULL), (dict(Y=None), NULL), (dict(dY=None), NULL), (dict(weights=None), NULL), (dict(dw=None), NULL),
    (dict(dO=A + 8), LAYOUT), (dict(Y=A + 2), LAYOUT), (dict(dY=A + 2), LAYOUT), (dict(weights=A + 2), LAYOUT),
    (dict(dw=A + 2), LAYOUT), (dict(lddo=56), LAYOUT), (dict(ldy=68), LAYOUT), (dict(lddy=56), LAYOUT)])
def test_gradient_refusals(kw, status):
    assert grad(**kw) == status


def test_exchange_empty_calls():
    assert gather(tokens=0, X=None, Y=None, position=None) == q.QGEMM_OK
    assert gather(rows=0, X=None, Y=None, position=None) == q.QGEMM_OK
    assert combine(tokens=0, Y=None, O=None, position=None) == q.QGEMM_OK
    assert grad(tokens=0, dO=None, Y=None, dY=None, position=None, weights=None, dw=None) == q.QGEMM_OK


QUANT = ["i8_rowwise", "f8_pertoken", "f8_block", "mx"]


@pytest.mark.parametrize("name", QUANT)
@pytest.mark.parametrize("kw,status", [
    (dict(X=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL), (dict(M=-1), SHAPE), (dict(I=0), SHAPE),
    (dict(I=120), SHAPE), (dict(M=1 << 31), SHAPE), (dict(I=1 << 30), SHAPE), (dict(X=A + 8), LAYOUT),
    (dict(ldx=248), LAYOUT), (dict(ldx=260), LAYOUT), (dict(count=A + 2), LAYOUT), (dict(Q=A + 8), LAYOUT),
    (dict(ldq=112, I=256, ldx=512), LAYOUT), (dict(ldq=136), LAYOUT)])
def test_swiglu_refusals(name, kw, status):
    assert swiglu(name, **kw) == status
    assert q.lib().qgemm_last_error()


@pytest.mark.parametrize("name", QUANT)
@pytest.mark.parametrize("kw,status", [
    (dict(norm=None), NULL), (dict(Y=None), NULL), (dict(R=None), NULL), (dict(gamma_post=None), NULL),
    (dict(gamma=None), NULL), (dict(Q=None), NULL), (dict(S=None), NULL), (dict(M=-1), SHAPE), (dict(K=0), SHAPE),
    (dict(K=120), SHAPE), (dict(M=1 << 31), SHAPE), (dict(K=1 << 31), SHAPE), (dict(eps=-1.0), SHAPE),
    (dict(eps=float("nan")), SHAPE), (dict(alpha=float("nan")), SHAPE), (dict(alpha=float("inf")), SHAPE),
    (dict(Y=A + 8), LAYOUT), (dict(R=A + 2), LAYOUT), (dict(Rout=A + 2), LAYOUT), (dict(gamma_post=A + 4), LAYOUT),
    (dict(gate=A + 4), LAYOUT), (dict(gamma=A + 4), LAYOUT), (dict(ldy=120), LAYOUT), (dict(ldr=132), LAYOUT),
    (dict(ldo=64), LAYOUT), (dict(Q=A + 8), LAYOUT), (dict(ldq=136), LAYOUT)])
def test_postnorm_refusals(name, kw, status):
    assert postnorm(name, **kw) == status
    assert q.lib().qgemm_last_error()


@pytest.mark.parametrize("f", [swiglu, postnorm])
def test_quantised_output_refusals_by_kind(f):
    wide = dict(I=96, ldx=256) if f is swiglu else dict(K=96)
    assert f("f8_block", **wide) == SHAPE
    assert f("f8_block", lds=0) == LAYOUT and f("mx", lds=3) == LAYOUT
    assert f("mx", fmt=2) == FORMAT
    assert f("f8_pertoken", S=A + 2) == LAYOUT


GROUPED = ["i8_rowwise", "f8_pertoken", "f8_blockscale", "mx"]


@pytest.mark.parametrize("name", GROUPED)
@pytest.mark.parametrize("kw,status", [
    (dict(A=None), NULL), (dict(B=None), NULL), (dict(sa=None), NULL), (dict(sb=None), NULL), (dict(C_=None), NULL),
    (dict(offsets=None), NULL), (dict(experts=0), SHAPE), (dict(experts=1025), SHAPE), (dict(a_rows=-1), SHAPE),
    (dict(a_rows=0), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=1 << 30), SHAPE), (dict(N=-1), SHAPE),
    (dict(N=1 << 31), SHAPE), (dict(K=0), SHAPE), (dict(K=192), SHAPE), (dict(K=1 << 31), SHAPE), (dict(top_k=0), SHAPE),
    (dict(top_k=65), SHAPE), (dict(order=None), SHAPE), (dict(A=A + 8), LAYOUT), (dict(B=B + 8), LAYOUT),
    (dict(lda=240), LAYOUT), (dict(ldb=240), LAYOUT), (dict(lda=264), LAYOUT), (dict(ldb=1 << 23), LAYOUT),
    (dict(a_rows=1 << 20, lda=2048), LAYOUT), (dict(sa=C + 2), LAYOUT), (dict(sb=D + 2), LAYOUT), (dict(bias=A + 1), LAYOUT),
    (dict(C_=A + 8), LAYOUT), (dict(ldc=56), LAYOUT), (dict(ldc=68), LAYOUT), (dict(ldc=1 << 22), LAYOUT),
    (dict(offsets=E + 2), LAYOUT), (dict(order=F + 2), LAYOUT), (dict(rows=(1 << 30) - 1, N=1 << 16, ldc=1 << 16), SHAPE)])
def test_grouped_refusals(name, kw, status):
    assert grouped(name, **kw) == status
    assert q.lib().qgemm_last_error()


def test_grouped_refusals_by_kind():
    assert grouped("mx", fmt=2) == FORMAT and grouped("mx", fmt=3) == FORMAT
    assert grouped("i8_rowwise", K=131072, lda=131072, ldb=131072) == SHAPE
    for name in ("f8_blockscale", "mx"):
        assert grouped(name, sa=C + 8) == LAYOUT and grouped(name, sb=D + 8) == LAYOUT


CALLS = [sort, gather, combine, grad, swiglu, postnorm] + [lambda n=n, **k: grouped(n, **k) for n in GROUPED]


@pytest.mark.parametrize("f", CALLS)
def test_device_and_launch_errors(f, monkeypatch):
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx1201")
    assert f() == q.QGEMM_ERR_UNSUPPORTED_DEVICE
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setenv("QGEMM_INJECT_LAUNCH_ERROR", "719")
    assert f() == q.QGEMM_ERR_HIP
    assert b"injected" in q.lib().qgemm_last_error()


@pytest.mark.parametrize("name", GROUPED)
def test_grouped_empty_calls(name):
    none = dict(A=None, B=None, sa=None, sb=None, offsets=None, C_=None)
    assert grouped(name, rows=0, **none) == q.QGEMM_OK
    assert grouped(name, N=0, **none) == q.QGEMM_OK


def test_norm_empty_calls():
    for name in QUANT:
        assert swiglu(name, M=0, X=None, Q=None, S=None) == q.QGEMM_OK
        assert postnorm(name, M=0, Y=None, R=None, gamma_post=None, gamma=None, Q=None, S=None) == q.QGEMM_OK
