"""The operators that a decoder layer runs between its GEMMs: argument
marshalling for the C entry points of the same names.  Errors as in the
package: ValueError for arguments, RuntimeError for the device."""
import ctypes
import struct

import torch

from . import (QGEMM_KV8_E4M3, QGEMM_KV8_I8, QGEMM_MX_E2M1, QGEMM_MX_E4M3, _check, _codes_out, lib)

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_empty = torch.empty
# (called with a tensor on the GPU: the runtime is up; a torch without GPUs has neither)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

# The compiled form of the expert operators' ordinary calls; without it, and for
# every call that is not ordinary, the functions below go the full way.
try:
    from . import _fast
    _fast.init(_current_device, _current_stream, _check)
except (ImportError, TypeError):
    _fast = None

# These calls stand between the GEMMs of a decode step, where the host's time is
# the step's: attributes are read once, and the device is changed only where it
# is not the current one.


def _enqueue(entry, device, stream, *args):
    """entry(*args, stream) on device; raises what it reports."""
    index = device.index
    if stream is None:
        stream = _current_stream(index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if _current_device() == index:
        status = entry(*args, stream)
    else:
        with torch.cuda.device(device):
            status = entry(*args, stream)
    if status:
        _check(status)


def _new(shape, dtype, device, stream, returned=True):
    """An uninitialised tensor that work on stream will write.  Memory of another
    stream's pool may still be in use by that stream's earlier work, so it
    comes from the given stream's own; what the caller gets is kept, once let go,
    until the current stream has used it too."""
    if stream is None:
        return _empty(shape, dtype=dtype, device=device)
    own = stream if isinstance(stream, torch.cuda.Stream) else \
        torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(own):
        t = _empty(shape, dtype=dtype, device=device)
    if returned:
        t.record_stream(current)
    return t


def _rows(t, name, dtypes=_BF16):
    """Shape and row stride (elements) of a 2-D GPU tensor with unit stride
    along its rows."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor of {dtypes}")
    shape, strides = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(shape)}")
    if strides[1] != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit stride along its rows")
    return shape, strides[0] if shape[0] > 1 else shape[1]


def _vec(t, name, n, device, dtypes=_BF16):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.device != device or t.numel() != n \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {dtypes} with {n} elements on {device}")
    return t.data_ptr()


# ------------------------------------------------------------ RMS norm

def _norm_common(X, gamma, residual, residual_out, stream):
    """What the four norms share: (shape, device, the arguments up to gamma,
    residual_out, its pointer and stride)."""
    shape, ldx = _rows(X, "X")
    device = X.device
    pr = ldr = po = ldo = 0
    if residual is not None:
        rshape, ldr = _rows(residual, "residual")
        if rshape != shape or residual.device != device:
            raise ValueError(f"residual must be {tuple(shape)} on {device}, got {tuple(rshape)} on {residual.device}")
        pr = residual.data_ptr()
        if residual_out is None:
            residual_out = _new(shape, torch.bfloat16, device, stream)
    if residual_out is not None:
        oshape, ldo = _rows(residual_out, "residual_out")
        if oshape != shape or residual_out.device != device:
            raise ValueError(f"residual_out must be {tuple(shape)} on {device}, got {tuple(oshape)} on "
                             f"{residual_out.device}")
        po = residual_out.data_ptr()
    return (shape, device, (X.data_ptr(), ldx, pr or None, ldr, _vec(gamma, "gamma", shape[1], device)),
            residual_out, po or None, ldo)


def _norm_codes(out, M, row, device, dtype, stream):
    """The codes' tensor and row stride in bytes."""
    if out is None:
        wide = row + (-row) % 16          # the library's rule for row strides
        out = _new((M, wide), dtype, device, stream)
        return (out if wide == row else out[:, :row]), wide
    if dtype is torch.int8:
        if not isinstance(out, torch.Tensor) or tuple(out.shape) != (M, row) or out.dtype != torch.int8 or out.device != device or (
                row > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be int8 [{M}, {row}] with unit stride along K on {device}")
    else:
        out = _codes_out(out, (M, row), device, "out")
    return out, out.stride(0) if M > 1 else row + (-row) % 16


def _norm_row(entry, dtype, X, gamma, eps, residual, residual_out, out, scale, stream):
    (M, K), device, head, residual_out, po, ldo = _norm_common(X, gamma, residual, residual_out, stream)
    out, ldq = _norm_codes(out, M, K, device, dtype, stream)
    if scale is None:
        scale = _new(M, torch.float32, device, stream)
        ps = scale.data_ptr()
    else:
        ps = _vec(scale, "scale", M, device, (torch.float32,))
    _enqueue(entry, device, stream, *head, eps, po, ldo, out.data_ptr(), ldq, ps, M, K)
    return out, scale, residual_out


def qgemm_rmsnorm_quant_i8_rowwise(X, gamma, eps=1e-6, residual=None, residual_out=None, out=None, scale=None,
                                   stream=None):
    """RMS norm of X + residual -> (int8 codes [M, K], scale fp32 [M], the sum
    in bf16): the A operand and scale_a of qgemm_i8_rowwise.  X, residual bf16
    [M, K], gamma bf16 [K]; residual_out may be residual itself; without a
    residual the third value is None unless residual_out is given."""
    return _norm_row(lib().qgemm_rmsnorm_quant_i8_rowwise, torch.int8, X, gamma, eps, residual, residual_out, out,
                     scale, stream)


def qgemm_rmsnorm_quant_f8_pertoken(X, gamma, eps=1e-6, residual=None, residual_out=None, out=None, scale=None,
                                    stream=None):
    """RMS norm of X + residual -> (e4m3 codes as uint8 [M, K], scale fp32
    [M], the sum in bf16): the A operand and scale_a of qgemm_f8_pertoken."""
    return _norm_row(lib().qgemm_rmsnorm_quant_f8_pertoken, torch.uint8, X, gamma, eps, residual, residual_out, out,
                     scale, stream)


def _norm_block(entry, first, row, parts, dtype, X, gamma, eps, residual, residual_out, out, scale, stream):
    (M, K), device, head, residual_out, po, ldo = _norm_common(X, gamma, residual, residual_out, stream)
    out, ldq = _norm_codes(out, M, row, device, torch.uint8, stream)
    if scale is None:
        scale, lds = _new((M, parts), dtype, device, stream), parts
    else:
        sshape, lds = _rows(scale, "scale", (dtype,))
        if tuple(sshape) != (M, parts) or scale.device != device:
            raise ValueError(f"scale must be {dtype} [{M}, {parts}] on {device}")
    _enqueue(entry, device, stream, *first, *head, eps, po, ldo, out.data_ptr(), ldq, scale.data_ptr(), lds, M, K)
    return out, scale, residual_out


def qgemm_rmsnorm_quant_f8_block(X, gamma, eps=1e-6, residual=None, residual_out=None, out=None, scale=None,
                                 stream=None):
    """RMS norm of X + residual -> (e4m3 codes as uint8 [M, K], scales fp32
    [M, K/128], the sum in bf16): the A operand and scale_a of
    qgemm_f8_blockscale.  K a multiple of 128."""
    K = _rows(X, "X")[0][1]
    if K % 128:
        raise ValueError(f"K={K} is not a multiple of 128")
    return _norm_block(lib().qgemm_rmsnorm_quant_f8_block, (), K, K // 128, torch.float32, X, gamma, eps, residual,
                       residual_out, out, scale, stream)


def qgemm_rmsnorm_quant_mx(fmt, X, gamma, eps=1e-6, residual=None, residual_out=None, out=None, scale=None,
                           stream=None):
    """RMS norm of X + residual -> (codes uint8 [M, K] (e4m3) or [M, K/2]
    (e2m1), ue8m0 scales uint8 [M, K/32], the sum in bf16): the A operand and
    scale_a of qgemm_mx."""
    if fmt not in (QGEMM_MX_E4M3, QGEMM_MX_E2M1):
        raise ValueError(f"unknown MX format {fmt}")
    K = _rows(X, "X")[0][1]
    return _norm_block(lib().qgemm_rmsnorm_quant_mx, (fmt,), K if fmt == QGEMM_MX_E4M3 else K // 2, K // 32,
                       torch.uint8, X, gamma, eps, residual, residual_out, out, scale, stream)


# ------------------------------------------------------------ norms after and before a block

# kinds of quantised output: MX format or -1, codes a byte, elements a scale
# covers (0: the row), int8 codes, ue8m0 scales
_I8_ROW, _F8_ROW, _F8_BLOCK = (-1, 1, 0, 1, 0), (-1, 1, 0, 0, 0), (-1, 1, 128, 0, 0)
_MX = {QGEMM_MX_E4M3: (QGEMM_MX_E4M3, 1, 32, 0, 1), QGEMM_MX_E2M1: (QGEMM_MX_E2M1, 2, 32, 0, 1)}

# qgemm_postnorm: Y, R, gamma_post, gate, gamma, Rout, their strides, eps, alpha
_POSTNORM = struct.Struct("@6P3q2f")


def _like(t, name, shape, device, dtypes=_BF16):
    """The row stride of a tensor that has to have this shape."""
    tshape, ld = _rows(t, name, dtypes)
    if tshape != shape or t.device != device:
        raise ValueError(f"{name} must be {tuple(shape)} on {device}, got {tuple(tshape)} on {t.device}")
    return ld


def _scales(scale, M, K, part, sdtype, device, stream):
    """(scale, the arguments that pass it on): one a row where part is 0, else
    one for each part elements."""
    if not part:
        if scale is None:
            scale = _new((M,), sdtype, device, stream)
            return scale, (scale.data_ptr(),)
        return scale, (_vec(scale, "scale", M, device, (sdtype,)),)
    parts = K // part
    if scale is None:
        scale = _new((M, parts), sdtype, device, stream)
        return scale, (scale.data_ptr(), parts)
    sshape, lds = _rows(scale, "scale", (sdtype,))
    if tuple(sshape) != (M, parts) or scale.device != device:
        raise ValueError(f"scale must be {sdtype} [{M}, {parts}] on {device}")
    return scale, (scale.data_ptr(), lds)


def _postnorm(name, kind, Y, residual, gamma_post, gamma, eps, gate, alpha, residual_out, out, scale, stream):
    """kind: (MX format or -1, codes a byte, elements a scale covers or 0 for
    the row, int8 codes, ue8m0 scales)."""
    L = lib()
    if _fast is not None and stream is None:
        got = _fast.postnorm(L.address[name], *kind, Y, residual, gamma_post, gamma, eps, gate, alpha, residual_out, out,
                             scale)
        if got is not None:
            return got
    fmt, per_byte, part, i8, ue8m0 = kind
    shape, ldy = _rows(Y, "Y")
    device = Y.device
    M, K = shape
    if K % (part or 32):
        raise ValueError(f"K={K} is not a multiple of {part or 32}")
    ldr = _like(residual, "residual", shape, device)
    if residual_out is None:
        residual_out, ldo = _new(shape, torch.bfloat16, device, stream), K
    else:
        ldo = _like(residual_out, "residual_out", shape, device)
    out, ldq = _norm_codes(out, M, K // per_byte, device, torch.int8 if i8 else torch.uint8, stream)
    scale, tail = _scales(scale, M, K, part, torch.uint8 if ue8m0 else torch.float32, device, stream)
    try:
        norm = _POSTNORM.pack(Y.data_ptr(), residual.data_ptr(), _vec(gamma_post, "gamma_post", K, device),
                              0 if gate is None else _vec(gate, "gate", K, device), _vec(gamma, "gamma", K, device),
                              residual_out.data_ptr(), ldy, ldr, ldo, eps, alpha)
    except (struct.error, OverflowError) as e:
        raise ValueError(f"eps={eps}, alpha={alpha}: {e}") from None
    _enqueue(getattr(L, name), device, stream, *((fmt,) if fmt >= 0 else ()), norm, out.data_ptr(), ldq, *tail, M, K)
    return out, scale, residual_out


def qgemm_postnorm_quant_i8_rowwise(Y, residual, gamma_post, gamma, eps=1e-6, gate=None, alpha=1.0, residual_out=None,
                                    out=None, scale=None, stream=None):
    """The end of a block and the beginning of the next: h = residual + alpha *
    gate * rmsnorm(Y; gamma_post), then the RMS norm of h with gamma -> (int8
    codes [M, K], scale fp32 [M], h in bf16).  Y, residual bf16 [M, K];
    gamma_post, gamma, gate (ones if None) bf16 [K]; residual_out may be
    residual itself."""
    return _postnorm("qgemm_postnorm_quant_i8_rowwise", _I8_ROW, Y, residual, gamma_post, gamma, eps, gate, alpha, residual_out,
                     out, scale, stream)


def qgemm_postnorm_quant_f8_pertoken(Y, residual, gamma_post, gamma, eps=1e-6, gate=None, alpha=1.0,
                                     residual_out=None, out=None, scale=None, stream=None):
    """The same -> (e4m3 codes as uint8 [M, K], scale fp32 [M], h in bf16)."""
    return _postnorm("qgemm_postnorm_quant_f8_pertoken", _F8_ROW, Y, residual, gamma_post, gamma, eps, gate, alpha, residual_out,
                     out, scale, stream)


def qgemm_postnorm_quant_f8_block(Y, residual, gamma_post, gamma, eps=1e-6, gate=None, alpha=1.0, residual_out=None,
                                  out=None, scale=None, stream=None):
    """The same -> (e4m3 codes as uint8 [M, K], scales fp32 [M, K/128], h in
    bf16).  K a multiple of 128."""
    return _postnorm("qgemm_postnorm_quant_f8_block", _F8_BLOCK, Y, residual, gamma_post, gamma, eps, gate, alpha, residual_out,
                     out, scale, stream)


def qgemm_postnorm_quant_mx(fmt, Y, residual, gamma_post, gamma, eps=1e-6, gate=None, alpha=1.0, residual_out=None,
                            out=None, scale=None, stream=None):
    """The same -> (codes uint8 [M, K] (e4m3) or [M, K/2] (e2m1), ue8m0 scales
    uint8 [M, K/32], h in bf16)."""
    if fmt not in (QGEMM_MX_E4M3, QGEMM_MX_E2M1):
        raise ValueError(f"unknown MX format {fmt}")
    return _postnorm("qgemm_postnorm_quant_mx", _MX[fmt], Y, residual, gamma_post, gamma, eps, gate, alpha, residual_out,
                     out, scale, stream)


# ------------------------------------------------------------ 8-bit cache

class _CacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block", ctypes.c_int32), ("fmt", ctypes.c_int32)]


class KV8Cache:
    """A paged cache of keys and values in 8 bits with one fp32 scale for each
    block of tokens and kv head.

        k        [blocks, kv_heads, block, head_dim]  int8, or e4m3 as
                 float8_e4m3fn or uint8
        v        [blocks, kv_heads, head_dim, block]  the same type
        k_scale, v_scale   fp32 [blocks, kv_heads]

    all contiguous on one device.  The cache holds the tensors; what is written
    into them is seen by the next call."""

    def __init__(self, k, v, k_scale, v_scale):
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous() or t.device != k.device:
                raise ValueError(f"{name} must be a contiguous tensor on a GPU device, the same for all four")
        if k.dim() != 4 or k.dtype not in (torch.int8, torch.uint8, torch.float8_e4m3fn) or v.dtype != k.dtype:
            raise ValueError("k and v must be 4-D, both int8 or both e4m3 (float8_e4m3fn or uint8)")
        blocks, heads, block, dim = k.shape
        if tuple(v.shape) != (blocks, heads, dim, block):
            raise ValueError(f"v must be {(blocks, heads, dim, block)} for k of {tuple(k.shape)}, got {tuple(v.shape)}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != torch.float32 or tuple(t.shape) != (blocks, heads):
                raise ValueError(f"{name} must be float32 {(blocks, heads)}, got {t.dtype} {tuple(t.shape)}")
        if dim not in (64, 128, 192, 256) or block not in (16, 32, 64, 128):
            raise ValueError(f"head_dim {dim} must be 64, 128, 192 or 256 and block {block} 16, 32, 64 or 128")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_blocks, self.kv_heads, self.block, self.head_dim = blocks, heads, block, dim
        self.fmt = QGEMM_KV8_I8 if k.dtype == torch.int8 else QGEMM_KV8_E4M3
        self.device = k.device
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), blocks, heads,
                                    dim, block, self.fmt)
        self._ref = ctypes.addressof(self._struct)

    @classmethod
    def empty(cls, num_blocks, kv_heads, head_dim, block=64, fmt=QGEMM_KV8_E4M3, device="cuda"):
        """A cache with nothing in it (contents undefined until appended)."""
        if fmt not in (QGEMM_KV8_E4M3, QGEMM_KV8_I8):
            raise ValueError(f"unknown cache format {fmt}")
        dtype = torch.int8 if fmt == QGEMM_KV8_I8 else torch.float8_e4m3fn
        return cls(torch.empty((num_blocks, kv_heads, block, head_dim), dtype=dtype, device=device),
                   torch.empty((num_blocks, kv_heads, head_dim, block), dtype=dtype, device=device),
                   torch.empty((num_blocks, kv_heads), dtype=torch.float32, device=device),
                   torch.empty((num_blocks, kv_heads), dtype=torch.float32, device=device))


def _cache(cache):
    """The cache's device."""
    if not isinstance(cache, KV8Cache):
        raise ValueError(f"cache must be a KV8Cache, got {type(cache).__name__}")
    return cache.device


def _token_rows(t, name, heads, dim, device, dtypes=_BF16):
    """Shape and token stride (elements) of a [tokens, heads, dim] tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.device != device:
        raise ValueError(f"{name} must be a tensor of {dtypes} on {device}")
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim}], got {tuple(shape)}")
    if st[2] != 1 or (shape[1] > 1 and st[1] != dim):
        raise ValueError(f"{name} must have unit stride along its last axis and adjacent heads")
    return shape, st[0] if shape[0] > 1 else shape[1] * dim


def _sequences(table, cu, lens, device):
    """(table pointer, stride, width), cu pointer, lens pointer, batch."""
    i32 = torch.int32
    if not (isinstance(table, torch.Tensor) and isinstance(cu, torch.Tensor) and isinstance(lens, torch.Tensor)):
        raise ValueError("block_table, cu_seqlens and kv_lens must be tensors")
    if table.dtype != i32 or cu.dtype != i32 or lens.dtype != i32 or table.device != device or cu.device != device \
            or lens.device != device:
        raise ValueError(f"block_table, cu_seqlens and kv_lens must be int32 on {device}")
    batch, tshape, tstride = lens.numel(), table.shape, table.stride()
    if lens.dim() != 1 or cu.dim() != 1 or cu.numel() != batch + 1 or not lens.is_contiguous() \
            or not cu.is_contiguous():
        raise ValueError(f"kv_lens must be [batch] and cu_seqlens [batch + 1], contiguous; got {tuple(lens.shape)} and "
                         f"{tuple(cu.shape)}")
    if len(tshape) != 2 or tshape[0] != batch or (tshape[1] > 1 and tstride[1] != 1):
        raise ValueError(f"block_table must be [{batch}, blocks] with unit stride along its rows, got {tuple(tshape)}")
    width = tshape[1]
    ldt = tstride[0] if batch > 1 else width
    if ldt < width:
        raise ValueError(f"block_table rows must not overlap: stride {ldt}, {width} entries")
    return table.data_ptr(), ldt, width, cu.data_ptr(), lens.data_ptr(), batch


def qgemm_kv8_append(cache, K, V, block_table, cu_seqlens, kv_lens, max_q, stream=None):
    """Append new tokens' keys and values to their sequences, quantised into
    the cache in place.  K, V bf16 [tokens, kv_heads, head_dim] (token rows may
    be slices of a wider row); block_table int32 [batch, blocks]; cu_seqlens
    int32 [batch + 1] the offsets of each sequence's new tokens; kv_lens int32
    [batch] the lengths with them; max_q at least the most new tokens of a
    sequence."""
    device = _cache(cache)
    kshape, ldk = _token_rows(K, "K", cache.kv_heads, cache.head_dim, device)
    vshape, ldv = _token_rows(V, "V", cache.kv_heads, cache.head_dim, device)
    if vshape != kshape:
        raise ValueError(f"K holds {kshape[0]} tokens, V {vshape[0]}")
    pt, ldt, width, pc, pl, batch = _sequences(block_table, cu_seqlens, kv_lens, device)
    _enqueue(lib().qgemm_kv8_append, device, stream, cache._ref, K.data_ptr(), ldk, V.data_ptr(), ldv, pt, ldt, width,
             pc, pl, kshape[0], batch, max_q)


def qgemm_kv8_attention(cache, Q, block_table, cu_seqlens, kv_lens, max_q, max_kv, sm_scale=None, causal=True,
                        window=0, out=None, workspace=None, stream=None):
    """Attention of the new tokens (already appended) over the cache -> bf16
    [tokens, heads, head_dim].  Q bf16 [tokens, heads, head_dim]; block_table,
    cu_seqlens, kv_lens, max_q as for qgemm_kv8_append; max_kv at least the
    longest kv_lens; sm_scale defaults to head_dim ** -0.5; window > 0 keeps
    the last that many positions of each token.  workspace: a uint8 tensor of
    at least qgemm_kv8_attention_workspace(...) bytes, allocated here if not
    given.  Tokens of no sequence are left as they are in ``out``."""
    device = _cache(cache)
    shape, ldq = _token_rows(Q, "Q", None, cache.head_dim, device)
    tokens, heads, dim = shape
    pt, ldt, width, pc, pl, batch = _sequences(block_table, cu_seqlens, kv_lens, device)
    if out is None:
        out, ldo = _new(shape, torch.bfloat16, device, stream), heads * dim
    else:
        oshape, ldo = _token_rows(out, "out", heads, dim, device, (torch.bfloat16,))
        if oshape != shape:
            raise ValueError(f"out must be bfloat16 {tuple(shape)}")
    if sm_scale is None:
        sm_scale = dim ** -0.5
    causal = 1 if causal else 0
    L = lib()
    pw = nbytes = 0
    if workspace is None:
        nbytes = L.qgemm_kv8_attention_workspace(cache._ref, tokens, batch, heads, max_q, max_kv, causal, window)
        if nbytes > 0:
            # let go here, it goes back to the stream that uses it
            workspace = _new(nbytes, torch.uint8, device, stream, returned=False)
            pw = workspace.data_ptr()
    elif not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    else:
        pw, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _enqueue(L.qgemm_kv8_attention, device, stream, cache._ref, Q.data_ptr(), ldq, pt, ldt, width, pc, pl, tokens,
             batch, heads, max_q, max_kv, sm_scale, causal, window, out.data_ptr(), ldo, pw or None, nbytes)
    return out


# ------------------------------------------------------------ 4-bit matvec

def _w4_args(X, W, bias, out, stream):
    (M, K), ldx = _rows(X, "X")
    (N, row), ldw = _rows(W, "W", (torch.uint8,))
    if row * 2 != K:
        raise ValueError(f"X is [M, K={K}] but W holds {2 * row} weights a row")
    device = X.device
    if W.device != device:
        raise ValueError(f"W must be on {device}, found on {W.device}")
    pb = None if bias is None else _vec(bias, "bias", N, device)
    if out is None:
        out, ldy = _new((M, N), torch.bfloat16, device, stream), N
    else:
        oshape, ldy = _rows(out, "out", (torch.bfloat16,))
        if tuple(oshape) != (M, N) or out.device != device:
            raise ValueError(f"out must be bfloat16 [{M}, {N}] with unit stride along N on {device}")
    return device, X.data_ptr(), ldx, W.data_ptr(), ldw if N > 1 else row + (-row) % 16, M, N, K, pb, out, ldy


def _w4_table(t, name, shape, dtypes, device):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be {dtypes} {shape}, contiguous, on {device}")
    return t.data_ptr()


def qgemm_w4_matvec_i4(X, W, scales, zeros=None, bias=None, out=None, stream=None):
    """bf16 X [M, K] (M <= 64) times int4 weights W uint8 [N, K/2] with bf16
    scales and uint8 zero points (8 where None) per group: both
    [N, K/group], group 32, 64 or 128 -> bf16 [M, N]."""
    device, px, ldx, pw, ldw, M, N, K, pb, out, ldy = _w4_args(X, W, bias, out, stream)
    groups = scales.shape[1] if isinstance(scales, torch.Tensor) and scales.dim() == 2 else 0
    if groups == 0 or K % groups:
        raise ValueError(f"scales must be a tensor [{N}, K/group] for K={K}, got {getattr(scales, 'shape', scales)}")
    ps = _w4_table(scales, "scales", (N, groups), _BF16, device)
    pz = None if zeros is None else _w4_table(zeros, "zeros", (N, groups), (torch.uint8,), device)
    _enqueue(lib().qgemm_w4_matvec_i4, device, stream, px, ldx, pw, ldw, ps, pz, K // groups, pb, out.data_ptr(), ldy,
             M, N, K)
    return out


_UE8M0 = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())


def qgemm_w4_matvec_mx(X, W, scale_b, b_layout, bias=None, out=None, stream=None):
    """bf16 X [M, K] (M <= 64) times the MXFP4 B operand of qgemm_mx: W uint8
    [N, K/2] e2m1, scale_b ue8m0 [N, K/32] (b_layout 1) or [ceil(N/32), K/32]
    (b_layout 32) -> bf16 [M, N]."""
    device, px, ldx, pw, ldw, M, N, K, pb, out, ldy = _w4_args(X, W, bias, out, stream)
    rows = -(-N // b_layout) if b_layout in (1, 32) else N
    ps = _w4_table(scale_b, "scale_b", (rows, K // 32), _UE8M0, device)
    _enqueue(lib().qgemm_w4_matvec_mx, device, stream, px, ldx, pw, ldw, ps, b_layout, pb, out.data_ptr(), ldy, M, N,
             K)
    return out
