"""The decoder-layer entry points on the CPU: bad arguments are refused with
the documented status before any HIP call (fake device pointers that nothing
dereferences), empty calls are no-ops, a wrong device is named."""
import ctypes as c

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


# ------------------------------------------------------------ 8-bit cache

class Struct(c.Structure):
    _fields_ = [("k", c.c_void_p), ("v", c.c_void_p), ("k_scale", c.c_void_p), ("v_scale", c.c_void_p),
                ("num_blocks", c.c_int64), ("kv_heads", c.c_int32), ("head_dim", c.c_int32), ("block", c.c_int32),
                ("fmt", c.c_int32)]


def cache(**kw):
    d = dict(k=A, v=B, k_scale=C, v_scale=D, num_blocks=10, kv_heads=2, head_dim=64, block=16, fmt=0)
    d.update(kw)
    return Struct(**d)


CACHE_BAD = [
    (dict(k=None), q.QGEMM_ERR_NULL_POINTER), (dict(v_scale=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(k=A + 8), q.QGEMM_ERR_BAD_LAYOUT), (dict(k_scale=C + 2), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(num_blocks=0), q.QGEMM_ERR_BAD_SHAPE), (dict(num_blocks=1 << 31), q.QGEMM_ERR_BAD_SHAPE),
    (dict(kv_heads=0), q.QGEMM_ERR_BAD_SHAPE), (dict(head_dim=96), q.QGEMM_ERR_BAD_SHAPE),
    (dict(block=48), q.QGEMM_ERR_BAD_SHAPE), (dict(fmt=2), q.QGEMM_ERR_BAD_FORMAT)]
SEQ_BAD = [
    (dict(table=None), q.QGEMM_ERR_NULL_POINTER), (dict(cu=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(lens=None), q.QGEMM_ERR_NULL_POINTER), (dict(table=E + 2), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(batch=-1), q.QGEMM_ERR_BAD_SHAPE), (dict(batch=65536), q.QGEMM_ERR_BAD_SHAPE),
    (dict(max_q=6), q.QGEMM_ERR_BAD_SHAPE), (dict(max_q=-1), q.QGEMM_ERR_BAD_SHAPE),
    (dict(tokens=1 << 31), q.QGEMM_ERR_BAD_SHAPE), (dict(width=9), q.QGEMM_ERR_BAD_SHAPE)]


def append(ref="ok", K=A, ldk=128, V=B, ldv=128, table=E, ldt=8, width=8, cu=E, lens=E, tokens=5, batch=2, max_q=3,
           **kw):
    ref = c.byref(cache(**kw)) if ref == "ok" else ref
    return q.lib().qgemm_kv8_append(ref, K, ldk, V, ldv, table, ldt, width, cu, lens, tokens, batch, max_q, None)


def attend(ref="ok", Q=A, ldq=512, table=E, ldt=8, width=8, cu=E, lens=E, tokens=5, batch=2, heads=8, max_q=3,
           max_kv=100, scale=0.125, causal=1, window=0, O=B, ldo=512, ws=None, nbytes=0, **kw):
    ref = c.byref(cache(**kw)) if ref == "ok" else ref
    return q.lib().qgemm_kv8_attention(ref, Q, ldq, table, ldt, width, cu, lens, tokens, batch, heads, max_q, max_kv,
                                       scale, causal, window, O, ldo, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", CACHE_BAD + SEQ_BAD + [
    (dict(ref=None), q.QGEMM_ERR_NULL_POINTER), (dict(K=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(V=None), q.QGEMM_ERR_NULL_POINTER), (dict(K=A + 8), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(ldk=120), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldv=132), q.QGEMM_ERR_BAD_LAYOUT)])
def test_append_refusals(kw, status):
    assert append(**kw) == status


@pytest.mark.parametrize("kw,status", CACHE_BAD + SEQ_BAD + [
    (dict(ref=None), q.QGEMM_ERR_NULL_POINTER), (dict(Q=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(O=None), q.QGEMM_ERR_NULL_POINTER), (dict(O=B + 8), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(ldq=508), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldo=504), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(heads=7), q.QGEMM_ERR_BAD_SHAPE), (dict(heads=0), q.QGEMM_ERR_BAD_SHAPE),
    (dict(max_kv=-1), q.QGEMM_ERR_BAD_SHAPE), (dict(max_kv=1 << 31), q.QGEMM_ERR_BAD_SHAPE),
    (dict(window=-1), q.QGEMM_ERR_BAD_SHAPE), (dict(window=5, causal=0), q.QGEMM_ERR_BAD_SHAPE),
    (dict(scale=float("nan")), q.QGEMM_ERR_BAD_SHAPE), (dict(scale=float("inf")), q.QGEMM_ERR_BAD_SHAPE)])
def test_attention_refusals(kw, status):
    assert attend(**kw) == status


def test_cache_empty_calls_and_device(monkeypatch):
    assert append(batch=0, table=None, cu=None, lens=None, K=None) == q.QGEMM_OK
    assert append(max_q=0, tokens=0, table=None, cu=None, lens=None, K=None) == q.QGEMM_OK
    assert attend(batch=0, table=None, cu=None, lens=None, Q=None) == q.QGEMM_OK
    assert attend(max_q=0, tokens=0, table=None, cu=None, lens=None, Q=None) == q.QGEMM_OK
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx1201")
    assert append() == q.QGEMM_ERR_UNSUPPORTED_DEVICE and attend() == q.QGEMM_ERR_UNSUPPORTED_DEVICE
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setenv("QGEMM_INJECT_LAUNCH_ERROR", "719")
    assert append() == q.QGEMM_ERR_HIP and attend() == q.QGEMM_ERR_HIP


def test_attention_workspace():
    size = q.lib().qgemm_kv8_attention_workspace
    k = cache(head_dim=128, block=64)
    assert size(c.byref(k), 5, 2, 8, 3, 100, 1, 0) == 0              # one short split
    need = size(c.byref(k), 1, 1, 8, 1, 100000, 1, 0)
    rows = 8 * (128 + 2) * 4
    assert need > 0 and need % rows == 0
    assert attend(head_dim=128, ldq=1024, ldo=1024, tokens=1, batch=1, max_q=1, max_kv=100000) == q.QGEMM_ERR_NULL_POINTER
    assert attend(head_dim=128, ldq=1024, ldo=1024, tokens=1, batch=1, max_q=1, max_kv=100000, ws=A,
                  nbytes=need - 1) == q.QGEMM_ERR_BAD_LAYOUT
    assert attend(head_dim=128, ldq=1024, ldo=1024, tokens=1, batch=1, max_q=1, max_kv=100000, ws=A + 4,
                  nbytes=need) == q.QGEMM_ERR_BAD_LAYOUT
    assert size(None, 1, 1, 8, 1, 100, 1, 0) == -1
    assert size(c.byref(k), 1, 1, 7, 1, 100, 1, 0) == -1
    assert size(c.byref(k), 1, 1, 8, 2, 100, 1, 0) == -1


# ------------------------------------------------------------ 4-bit matvec

def i4(X=A, ldx=256, W=B, ldw=128, S=C, Z=D, group=64, bias=E, Y=E, ldy=32, M=2, N=32, K=256):
    return q.lib().qgemm_w4_matvec_i4(X, ldx, W, ldw, S, Z, group, bias, Y, ldy, M, N, K, None)


def mx(X=A, ldx=256, W=B, ldw=128, S=C, layout=1, bias=E, Y=E, ldy=32, M=2, N=32, K=256):
    return q.lib().qgemm_w4_matvec_mx(X, ldx, W, ldw, S, layout, bias, Y, ldy, M, N, K, None)


@pytest.mark.parametrize("f", [i4, mx])
@pytest.mark.parametrize("kw,status", [
    (dict(X=None), q.QGEMM_ERR_NULL_POINTER), (dict(W=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(S=None), q.QGEMM_ERR_NULL_POINTER), (dict(Y=None), q.QGEMM_ERR_NULL_POINTER),
    (dict(M=-1), q.QGEMM_ERR_BAD_SHAPE), (dict(M=65), q.QGEMM_ERR_BAD_SHAPE), (dict(N=-1), q.QGEMM_ERR_BAD_SHAPE),
    (dict(K=0), q.QGEMM_ERR_BAD_SHAPE), (dict(K=240), q.QGEMM_ERR_BAD_SHAPE), (dict(N=1 << 31), q.QGEMM_ERR_BAD_SHAPE),
    (dict(X=A + 8), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldx=252), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(W=B + 4), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldw=112), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(ldw=136), q.QGEMM_ERR_BAD_LAYOUT), (dict(bias=E + 1), q.QGEMM_ERR_BAD_LAYOUT),
    (dict(Y=E + 1), q.QGEMM_ERR_BAD_LAYOUT), (dict(ldy=31), q.QGEMM_ERR_BAD_LAYOUT)])
def test_matvec_refusals(f, kw, status):
    assert f(**kw) == status


def test_matvec_refusals_by_kind_empty_and_device(monkeypatch):
    assert i4(group=16) == q.QGEMM_ERR_BAD_SHAPE and i4(group=0) == q.QGEMM_ERR_BAD_SHAPE
    assert i4(S=C + 1) == q.QGEMM_ERR_BAD_LAYOUT
    assert mx(layout=2) == q.QGEMM_ERR_BAD_FORMAT
    for f in (i4, mx):
        assert f(M=0, X=None, W=None, S=None, Y=None) == q.QGEMM_OK
        assert f(N=0, X=None, W=None, S=None, Y=None) == q.QGEMM_OK
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx1201")
    assert i4() == q.QGEMM_ERR_UNSUPPORTED_DEVICE and mx() == q.QGEMM_ERR_UNSUPPORTED_DEVICE
    monkeypatch.setenv("QGEMM_FAKE_ARCH", "gfx950")
    monkeypatch.setenv("QGEMM_INJECT_LAUNCH_ERROR", "719")
    assert i4() == q.QGEMM_ERR_HIP and mx() == q.QGEMM_ERR_HIP


def test_attention_limits_are_named():
    for kw in (dict(max_q=1 << 24, tokens=1 << 24), dict(max_q=1 << 23, tokens=1 << 23, heads=16, ldq=1024, ldo=1024)):
        assert attend(**kw, ws=A, nbytes=1 << 60) == q.QGEMM_ERR_BAD_SHAPE
        assert b"max_q" in q.lib().qgemm_last_error()
