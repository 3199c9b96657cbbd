"""The operators that a decoder layer runs between its GEMMs: argument
marshalling for the C entry points of the same names.  Errors as in the
package: ValueError for arguments, RuntimeError for the device."""
import ctypes

import torch

from . import (QGEMM_KV8_E4M3, QGEMM_KV8_I8, QGEMM_MX_E2M1, QGEMM_MX_E4M3, _check, _codes_out, _ld_bytes, _operand, _ptr, _same_device, _stream,
               _vector, lib)

_BF16 = (torch.bfloat16, torch.int16, torch.uint16)


# ------------------------------------------------------------ RMS norm

def _bf16_rows(t, name, shape, device):
    if t is None:
        return 0
    ld = _operand(t, name, _BF16) // 2
    if tuple(t.shape) != shape or t.device != device:
        raise ValueError(f"{name} must be [{shape[0]}, {shape[1]}] on {device}, got {tuple(t.shape)} on {t.device}")
    return ld


def _norm_args(X, gamma, residual, residual_out):
    """The tensors and strides common to the four norms."""
    ldx = _operand(X, "X", _BF16) // 2
    shape, device = tuple(X.shape), X.device
    ldr = _bf16_rows(residual, "residual", shape, device)
    if residual is not None and residual_out is None:
        residual_out = torch.empty(shape, dtype=torch.bfloat16, device=device)
    ldo = _bf16_rows(residual_out, "residual_out", shape, device)
    _vector(gamma, "gamma", shape[1], _BF16)
    _same_device(device, gamma)
    return ldx, ldr, ldo, residual_out


def _norm_row(entry, code_dtype, X, gamma, eps, residual, residual_out, out, scale, stream):
    ldx, ldr, ldo, residual_out = _norm_args(X, gamma, residual, residual_out)
    M, K = X.shape
    if code_dtype is torch.int8:
        if out is None:
            out = torch.empty((M, K + (-K) % 16), dtype=torch.int8, device=X.device)[:, :K]
        elif tuple(out.shape) != (M, K) or out.dtype != torch.int8 or (K > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be int8 [{M}, {K}] with unit stride along K")
    else:
        out = _codes_out(out, (M, K), X.device, "out")
    if scale is None:
        scale = torch.empty(M, dtype=torch.float32, device=X.device)
    _vector(scale, "scale", M, (torch.float32,))
    _same_device(X.device, out, scale)
    with torch.cuda.device(X.device):
        _check(entry(_ptr(X), ldx, _ptr(residual), ldr, _ptr(gamma), eps, _ptr(residual_out), ldo, _ptr(out),
                     _ld_bytes(out, K), _ptr(scale), M, K, _stream(X.device, stream)))
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


def _norm_scales(scales, shape, dtype, device):
    if scales is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if (scales.dtype != dtype or tuple(scales.shape) != shape or scales.device != device
            or (shape[1] > 1 and scales.stride(1) != 1)):
        raise ValueError(f"scale must be {dtype} {shape} with unit stride along its rows on {device}")
    return scales


def qgemm_rmsnorm_quant_f8_block(X, gamma, eps=1e-6, residual=None, residual_out=None, out=None, scale=None,
                                 stream=None):
    """RMS norm of X + residual -> (e4m3 codes as uint8 [M, K], scales fp32
    [M, K/128], the sum in bf16): the A operand and scale_a of
    qgemm_f8_blockscale.  K a multiple of 128."""
    ldx, ldr, ldo, residual_out = _norm_args(X, gamma, residual, residual_out)
    M, K = X.shape
    if K % 128:
        raise ValueError(f"K={K} is not a multiple of 128")
    out = _codes_out(out, (M, K), X.device, "out")
    scale = _norm_scales(scale, (M, K // 128), torch.float32, X.device)
    lds = scale.stride(0) if M > 1 else K // 128
    with torch.cuda.device(X.device):
        _check(lib().qgemm_rmsnorm_quant_f8_block(_ptr(X), ldx, _ptr(residual), ldr, _ptr(gamma), eps,
                                                  _ptr(residual_out), ldo, _ptr(out), _ld_bytes(out, K), _ptr(scale),
                                                  lds, M, K, _stream(X.device, stream)))
    return out, scale, residual_out


def qgemm_rmsnorm_quant_mx(fmt, X, gamma, eps=1e-6, residual=None, residual_out=None, out=None, scale=None,
                           stream=None):
    """RMS norm of X + residual -> (codes uint8 [M, K] (e4m3) or [M, K/2]
    (e2m1), ue8m0 scales uint8 [M, K/32], the sum in bf16): the A operand and
    scale_a of qgemm_mx."""
    if fmt not in (QGEMM_MX_E4M3, QGEMM_MX_E2M1):
        raise ValueError(f"unknown MX format {fmt}")
    ldx, ldr, ldo, residual_out = _norm_args(X, gamma, residual, residual_out)
    M, K = X.shape
    row = K if fmt == QGEMM_MX_E4M3 else K // 2
    out = _codes_out(out, (M, row), X.device, "out")
    scale = _norm_scales(scale, (M, K // 32), torch.uint8, X.device)
    lds = scale.stride(0) if M > 1 else K // 32
    with torch.cuda.device(X.device):
        _check(lib().qgemm_rmsnorm_quant_mx(fmt, _ptr(X), ldx, _ptr(residual), ldr, _ptr(gamma), eps,
                                            _ptr(residual_out), ldo, _ptr(out), _ld_bytes(out, row), _ptr(scale), lds,
                                            M, K, _stream(X.device, stream)))
    return out, scale, residual_out


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


def _token_rows(t, name, heads, dim, device):
    """Token stride (elements) of a [tokens, heads, dim] bf16 tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype not in _BF16 or t.device != device:
        raise ValueError(f"{name} must be a bfloat16 tensor on {device}")
    shape, st = t.shape, t.stride()
    if len(shape) != 3 or (heads is not None and shape[1] != heads) or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads or 'heads'}, {dim}], got {tuple(shape)}")
    if st[2] != 1 or (shape[1] > 1 and st[1] != dim):
        raise ValueError(f"{name} must have unit stride along its last axis and adjacent heads")
    return st[0] if shape[0] > 1 else shape[1] * dim


def _sequences(table, cu, lens, device):
    batch = lens.shape[0]
    for name, t in (("block_table", table), ("cu_seqlens", cu), ("kv_lens", lens)):
        if t.dtype != torch.int32 or t.device != device:
            raise ValueError(f"{name} must be int32 on {device}, got {t.dtype} on {t.device}")
    if lens.dim() != 1 or cu.dim() != 1 or cu.shape[0] != batch + 1 or not lens.is_contiguous() \
            or not cu.is_contiguous():
        raise ValueError(f"kv_lens must be [batch] and cu_seqlens [batch + 1], contiguous; got {tuple(lens.shape)} and "
                         f"{tuple(cu.shape)}")
    if table.dim() != 2 or table.shape[0] != batch or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"block_table must be [{batch}, blocks] with unit stride along its rows, got "
                         f"{tuple(table.shape)}")
    width = table.shape[1]
    return batch, max(table.stride(0), width) if batch > 1 else width, width


def qgemm_kv8_append(cache, K, V, block_table, cu_seqlens, kv_lens, max_q, stream=None):
    """Append new tokens' keys and values to their sequences, quantised into
    the cache in place.  K, V bf16 [tokens, kv_heads, head_dim] (token rows may
    be slices of a wider row); block_table int32 [batch, blocks]; cu_seqlens
    int32 [batch + 1] the offsets of each sequence's new tokens; kv_lens int32
    [batch] the lengths with them; max_q at least the most new tokens of a
    sequence."""
    device = cache.device
    ldk = _token_rows(K, "K", cache.kv_heads, cache.head_dim, device)
    ldv = _token_rows(V, "V", cache.kv_heads, cache.head_dim, device)
    tokens = K.shape[0]
    if V.shape[0] != tokens:
        raise ValueError(f"K holds {tokens} tokens, V {V.shape[0]}")
    batch, ldt, width = _sequences(block_table, cu_seqlens, kv_lens, device)
    with torch.cuda.device(device):
        _check(lib().qgemm_kv8_append(cache._ref, _ptr(K), ldk, _ptr(V), ldv, _ptr(block_table), ldt, width,
                                      _ptr(cu_seqlens), _ptr(kv_lens), tokens, batch, max_q, _stream(device, stream)))


def qgemm_kv8_attention(cache, Q, block_table, cu_seqlens, kv_lens, max_q, max_kv, sm_scale=None, causal=True,
                        window=0, out=None, workspace=None, stream=None):
    """Attention of the new tokens (already appended) over the cache -> bf16
    [tokens, heads, head_dim].  Q bf16 [tokens, heads, head_dim]; block_table,
    cu_seqlens, kv_lens, max_q as for qgemm_kv8_append; max_kv at least the
    longest kv_lens; sm_scale defaults to head_dim ** -0.5; window > 0 keeps
    the last that many positions of each token.  workspace: a uint8 tensor of
    at least qgemm_kv8_attention_workspace(...) bytes, allocated here if not
    given.  Tokens of no sequence are left as they are in ``out``."""
    device = cache.device
    ldq = _token_rows(Q, "Q", None, cache.head_dim, device)
    tokens, heads = Q.shape[0], Q.shape[1]
    batch, ldt, width = _sequences(block_table, cu_seqlens, kv_lens, device)
    if out is None:
        out = torch.empty((tokens, heads, cache.head_dim), dtype=torch.bfloat16, device=device)
    elif out.dtype != torch.bfloat16 or out.shape[0] != tokens:
        raise ValueError(f"out must be bfloat16 [{tokens}, {heads}, {cache.head_dim}]")
    ldo = _token_rows(out, "out", heads, cache.head_dim, device)
    if sm_scale is None:
        sm_scale = cache.head_dim ** -0.5
    causal = 1 if causal else 0
    if workspace is None:
        need = lib().qgemm_kv8_attention_workspace(cache._ref, tokens, batch, heads, max_q, max_kv, causal, window)
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    with torch.cuda.device(device):
        _check(lib().qgemm_kv8_attention(cache._ref, _ptr(Q), ldq, _ptr(block_table), ldt, width, _ptr(cu_seqlens),
                                         _ptr(kv_lens), tokens, batch, heads, max_q, max_kv, sm_scale, causal, window,
                                         _ptr(out), ldo, _ptr(workspace), nbytes, _stream(device, stream)))
    return out


# ------------------------------------------------------------ 4-bit matvec

def _w4_args(X, W, bias, out):
    ldx = _operand(X, "X", _BF16) // 2
    ldw = _operand(W, "W", (torch.uint8,))
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] * 2 != K:
        raise ValueError(f"X is [M, K={K}] but W holds {2 * W.shape[1]} weights a row")
    device = X.device
    _vector(bias, "bias", N, _BF16)
    _same_device(device, W, bias)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=device)
    elif (tuple(out.shape) != (M, N) or out.dtype != torch.bfloat16 or out.device != device
          or (N > 1 and out.stride(1) != 1)):
        raise ValueError(f"out must be bfloat16 [{M}, {N}] with unit stride along N on {device}")
    return ldx, ldw if N > 1 else ldw + (-ldw) % 16, M, N, K, out, out.stride(0) if M > 1 else N


def _w4_table(t, name, shape, dtypes, device):
    if t.dtype not in dtypes or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be {dtypes} {shape}, contiguous, on {device}")


def qgemm_w4_matvec_i4(X, W, scales, zeros=None, bias=None, out=None, stream=None):
    """bf16 X [M, K] (M <= 64) times int4 weights W uint8 [N, K/2] with bf16
    scales and uint8 zero points (8 where None) per group: both
    [N, K/group], group 32, 64 or 128 -> bf16 [M, N]."""
    ldx, ldw, M, N, K, out, ldy = _w4_args(X, W, bias, out)
    groups = scales.shape[1] if scales.dim() == 2 else 0
    if groups == 0 or K % groups:
        raise ValueError(f"scales must be [{N}, K/group], got {tuple(scales.shape)} for K={K}")
    _w4_table(scales, "scales", (N, groups), _BF16, X.device)
    if zeros is not None:
        _w4_table(zeros, "zeros", (N, groups), (torch.uint8,), X.device)
    with torch.cuda.device(X.device):
        _check(lib().qgemm_w4_matvec_i4(_ptr(X), ldx, _ptr(W), ldw, _ptr(scales), _ptr(zeros), K // groups, _ptr(bias),
                                        _ptr(out), ldy, M, N, K, _stream(X.device, stream)))
    return out


def qgemm_w4_matvec_mx(X, W, scale_b, b_layout, bias=None, out=None, stream=None):
    """bf16 X [M, K] (M <= 64) times the MXFP4 B operand of qgemm_mx: W uint8
    [N, K/2] e2m1, scale_b ue8m0 [N, K/32] (b_layout 1) or [ceil(N/32), K/32]
    (b_layout 32) -> bf16 [M, N]."""
    ldx, ldw, M, N, K, out, ldy = _w4_args(X, W, bias, out)
    rows = -(-N // b_layout) if b_layout in (1, 32) else N
    sdt = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())
    _w4_table(scale_b, "scale_b", (rows, K // 32), sdt, X.device)
    with torch.cuda.device(X.device):
        _check(lib().qgemm_w4_matvec_mx(_ptr(X), ldx, _ptr(W), ldw, _ptr(scale_b), b_layout, _ptr(bias), _ptr(out),
                                        ldy, M, N, K, _stream(X.device, stream)))
    return out
