"""The operators that a decoder layer runs between its GEMMs: argument
marshalling for the C entry points of the same names.  Errors as in the
package: ValueError for arguments, RuntimeError for the device."""
import torch

from . import (QGEMM_MX_E2M1, QGEMM_MX_E4M3, _check, _codes_out, _ld_bytes, _operand, _ptr, _same_device, _stream,
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
