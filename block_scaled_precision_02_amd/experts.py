"""A layer of experts: the choices in order of experts, tokens' rows to the
experts and back with their gradients, the grouped GEMMs, and SwiGLU between
them.  Argument marshalling for the C entry points of the same names; errors as
in the package: ValueError for arguments, RuntimeError for the device."""
from operator import index

import torch

from . import QGEMM_MX_E2M1, QGEMM_MX_E4M3, lib
from .layer import (_BF16, _F8_BLOCK, _F8_ROW, _I8_ROW, _MX, _enqueue, _fast, _like, _new, _norm_codes, _rows, _scales,
                    _vec)

_I32 = torch.int32
_F32 = (torch.float32,)


def _out_rows(t, name, shape, device, stream):
    """(tensor, row stride) of a bf16 output, allocated where not given."""
    if t is None:
        return _new(shape, torch.bfloat16, device, stream), shape[1]
    return t, _like(t, name, shape, device, (torch.bfloat16,))


def _choices(t, name):
    """(tokens, top_k) of an int32 [tokens, top_k] tensor."""
    if not isinstance(t, torch.Tensor) or t.dtype != _I32 or not t.is_cuda or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 GPU tensor [tokens, top_k]")
    return t.shape


def _array(t, name, shape, dtype, device):
    """The address of a contiguous tensor that has to have this shape."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or t.shape != shape \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on {device}")
    return t.data_ptr()


def _count(v, name, most, least=1):
    try:
        n = index(v)
    except TypeError:
        n = least - 1
    if not least <= n <= most:
        raise ValueError(f"{name}={v}: need a whole number, {least} to {most}")
    return n


# ------------------------------------------------------------ sort and exchange

def qgemm_moe_sort(ids, experts, offsets=None, order=None, position=None, workspace=None, stream=None):
    """The choices ids int32 [tokens, top_k] in order of experts -> (offsets
    int32 [experts + 1], order int32 [tokens * top_k], position int32
    [tokens, top_k]): rows offsets[e] .. offsets[e+1]-1 are expert e's, row r is
    slot order[r] (token order[r] // top_k), slot s is row position[s].  Ids
    outside [0, experts) have no row (position -1; order -1 past the last row).
    workspace: a uint8 tensor of at least qgemm_moe_sort_workspace(...) bytes,
    allocated here if not given."""
    L = lib()
    if _fast is not None and stream is None and offsets is None and order is None and position is None \
            and workspace is None:
        got = _fast.moe_sort(L.address["qgemm_moe_sort"], L.address["qgemm_moe_sort_workspace"], ids, experts)
        if got is not None:
            return got
    tokens, top_k = _choices(ids, "ids")
    device = ids.device
    experts = _count(experts, "experts", 1024)
    slots = tokens * top_k
    if offsets is None:
        offsets = _new((experts + 1,), _I32, device, stream)
        po = offsets.data_ptr()
    else:
        po = _array(offsets, "offsets", (experts + 1,), _I32, device)
    if order is None:
        order = _new((slots,), _I32, device, stream)
        pr = order.data_ptr()
    else:
        pr = _array(order, "order", (slots,), _I32, device)
    if position is None:
        position = _new((tokens, top_k), _I32, device, stream)
        pp = position.data_ptr()
    else:
        pp = _array(position, "position", (tokens, top_k), _I32, device)
    pw = nbytes = 0
    if workspace is None:
        nbytes = L.qgemm_moe_sort_workspace(tokens, top_k, experts)
        if nbytes > 0:
            # let go here, it goes back to the stream that uses it
            workspace = _new(nbytes, torch.uint8, device, stream, returned=False)
            pw = workspace.data_ptr()
    elif not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    else:
        pw, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _enqueue(L.qgemm_moe_sort, device, stream, ids.data_ptr(), tokens, top_k, experts, po, pr, pp, pw or None, nbytes)
    return offsets, order, position


def _token_rows(t, name, tokens, device):
    shape, ld = _rows(t, name)
    if shape[0] != tokens or t.device != device:
        raise ValueError(f"{name} must have {tokens} rows on {device}, got {tuple(shape)} on {t.device}")
    return shape[1], ld


def qgemm_moe_gather(X, position, rows=None, out=None, stream=None):
    """Each token's row to the rows of its choices: out[position[t, j]] = X[t].
    X bf16 [tokens, H], position int32 [tokens, top_k] -> bf16 [rows, H] (rows:
    tokens * top_k unless given); rows that no slot takes are left as they are
    (in a new result: any values)."""
    L = lib()
    if _fast is not None and stream is None:
        got = _fast.moe_gather(L.address["qgemm_moe_gather"], X, position, rows, out)
        if got is not None:
            return got
    tokens, top_k = _choices(position, "position")
    device = position.device
    H, ldx = _token_rows(X, "X", tokens, device)
    if rows is not None:
        rows = _count(rows, "rows", (1 << 31) - 1, 0)
    elif out is not None:
        rows = _rows(out, "out", (torch.bfloat16,))[0][0]
    out, ldo = _out_rows(out, "out", (tokens * top_k if rows is None else rows, H), device, stream)
    _enqueue(L.qgemm_moe_gather, device, stream, X.data_ptr(), ldx, position.data_ptr(), out.data_ptr(), ldo,
             tokens, top_k, out.shape[0], H)
    return out


def qgemm_moe_combine(Y, position, weights=None, residual=None, out=None, stream=None):
    """The rows of each token's choices, summed: out[t] = residual[t] + sum_j
    weights[t, j] * Y[position[t, j]].  Y bf16 [rows, H], position int32
    [tokens, top_k], weights fp32 [tokens, top_k] (ones if None), residual bf16
    [tokens, H] (zeros if None; may be out) -> bf16 [tokens, H].  With neither
    it is the gradient of qgemm_moe_gather."""
    L = lib()
    if _fast is not None and stream is None:
        got = _fast.moe_combine(L.address["qgemm_moe_combine"], Y, position, weights, residual, out)
        if got is not None:
            return got
    tokens, top_k = _choices(position, "position")
    device = position.device
    (rows, H), ldy = _rows(Y, "Y")
    if Y.device != device:
        raise ValueError(f"Y must be on {device}, found on {Y.device}")
    pw = None if weights is None else _array(weights, "weights", (tokens, top_k), torch.float32, device)
    pr = ldr = 0
    if residual is not None:
        rH, ldr = _token_rows(residual, "residual", tokens, device)
        if rH != H:
            raise ValueError(f"residual must be [{tokens}, {H}], got [{tokens}, {rH}]")
        pr = residual.data_ptr()
    out, ldo = _out_rows(out, "out", (tokens, H), device, stream)
    _enqueue(L.qgemm_moe_combine, device, stream, Y.data_ptr(), ldy, position.data_ptr(), pw, pr or None, ldr,
             out.data_ptr(), ldo, tokens, top_k, rows, H)
    return out


def qgemm_moe_combine_grad(dout, Y, position, weights, dY=None, dweights=None, stream=None):
    """The gradient of qgemm_moe_combine: (dY bf16 [rows, H], dY[position[t, j]]
    = weights[t, j] * dout[t]; dweights fp32 [tokens, top_k], the product of
    dout[t] and Y[position[t, j]]).  Rows of dY that no slot takes are left as
    they are (in a new dY: any values); dY may be Y.  The residual's gradient is
    dout."""
    L = lib()
    if _fast is not None and stream is None:
        got = _fast.moe_combine_grad(L.address["qgemm_moe_combine_grad"], dout, Y, position, weights, dY, dweights)
        if got is not None:
            return got
    tokens, top_k = _choices(position, "position")
    device = position.device
    H, ldd = _token_rows(dout, "dout", tokens, device)
    (rows, yH), ldy = _rows(Y, "Y")
    if yH != H or Y.device != device:
        raise ValueError(f"Y must be [rows, {H}] on {device}, got {tuple(Y.shape)} on {Y.device}")
    pw = _array(weights, "weights", (tokens, top_k), torch.float32, device)
    dY, ldg = _out_rows(dY, "dY", (rows, H), device, stream)
    if dweights is None:
        dweights = _new((tokens, top_k), torch.float32, device, stream)
    _enqueue(L.qgemm_moe_combine_grad, device, stream, dout.data_ptr(), ldd, Y.data_ptr(), ldy,
             position.data_ptr(), pw, dY.data_ptr(), ldg, _array(dweights, "dweights", (tokens, top_k), torch.float32, device),
             tokens, top_k, rows, H)
    return dY, dweights


# ------------------------------------------------------------ SwiGLU

def _swiglu(name, kind, X, count, out, scale, stream):
    """kind: as for the norms (layer.py)."""
    L = lib()
    if _fast is not None and stream is None:
        got = _fast.swiglu(L.address[name], *kind, X, count, out, scale)
        if got is not None:
            return got
    fmt, per_byte, part, i8, ue8m0 = kind
    (M, wide), ldx = _rows(X, "X")
    I = wide // 2
    if wide % 2 or I % (part or 32):
        raise ValueError(f"X is [M, {wide}]: need two halves, each a multiple of {part or 32}")
    device = X.device
    pc = None if count is None else _vec(count, "count", 1, device, (_I32,))
    out, ldq = _norm_codes(out, M, I // per_byte, device, torch.int8 if i8 else torch.uint8, stream)
    scale, tail = _scales(scale, M, I, part, torch.uint8 if ue8m0 else torch.float32, device, stream)
    _enqueue(getattr(L, name), device, stream, *((fmt,) if fmt >= 0 else ()), X.data_ptr(), ldx, pc, out.data_ptr(), ldq, *tail, M, I)
    return out, scale


def qgemm_swiglu_quant_i8_rowwise(X, count=None, out=None, scale=None, stream=None):
    """silu(g) * u of X = [g | u], bf16 [M, 2 I] -> (int8 codes [M, I], scale
    fp32 [M]): the A operand and scale_a of qgemm_i8_rowwise and its grouped
    form.  count: int32 GPU tensor of one element (such as offsets[-1:] of the
    sort): rows from there on are left as they are."""
    return _swiglu("qgemm_swiglu_quant_i8_rowwise", _I8_ROW, X, count, out, scale, stream)


def qgemm_swiglu_quant_f8_pertoken(X, count=None, out=None, scale=None, stream=None):
    """silu(g) * u of X = [g | u] -> (e4m3 codes as uint8 [M, I], scale fp32
    [M]): the A operand and scale_a of qgemm_f8_pertoken and its grouped form;
    count as for the int8 form."""
    return _swiglu("qgemm_swiglu_quant_f8_pertoken", _F8_ROW, X, count, out, scale, stream)


def qgemm_swiglu_quant_f8_block(X, count=None, out=None, scale=None, stream=None):
    """silu(g) * u of X = [g | u] -> (e4m3 codes as uint8 [M, I], scales fp32
    [M, I/128]): the A operand and scale_a of qgemm_f8_blockscale and its
    grouped form.  I a multiple of 128."""
    return _swiglu("qgemm_swiglu_quant_f8_block", _F8_BLOCK, X, count, out, scale, stream)


def qgemm_swiglu_quant_mx(fmt, X, count=None, out=None, scale=None, stream=None):
    """silu(g) * u of X = [g | u] -> (codes uint8 [M, I] (e4m3) or [M, I/2]
    (e2m1), ue8m0 scales uint8 [M, I/32]): the A operand and scale_a of qgemm_mx
    and its grouped form."""
    if fmt not in (QGEMM_MX_E4M3, QGEMM_MX_E2M1):
        raise ValueError(f"unknown MX format {fmt}")
    return _swiglu("qgemm_swiglu_quant_mx", _MX[fmt], X, count, out, scale, stream)


# ------------------------------------------------------------ grouped GEMMs

_E4M3 = (torch.uint8, torch.float8_e4m3fn)
_UE8M0 = (torch.uint8,) + ((torch.float8_e8m0fnu,) if hasattr(torch, "float8_e8m0fnu") else ())


def _table(t, name, shape, dtypes, device):
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes or t.shape != shape or t.device != device \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be {dtypes} {tuple(shape)}, contiguous, on {device}")
    return t.data_ptr()


# name, MX format or -1, elements a byte, K elements a scale covers (0: the row),
# rows of B that a scale covers (0 with int8)
_G_I8 = ("qgemm_i8_rowwise_grouped", -1, 1, 0, 0)
_G_F8 = ("qgemm_f8_pertoken_grouped", -1, 1, 0, 1)
_G_BLOCK = ("qgemm_f8_blockscale_grouped", -1, 1, 128, 128)
_G_MX = {QGEMM_MX_E4M3: ("qgemm_mx_grouped", QGEMM_MX_E4M3, 1, 32, 1),
         QGEMM_MX_E2M1: ("qgemm_mx_grouped", QGEMM_MX_E2M1, 2, 32, 1)}


def _grouped(kind, A, B, scale_a, scale_b, offsets, order, top_k, bias, out, stream):
    L = lib()
    if _fast is not None and stream is None:
        got = _fast.grouped(L.address[kind[0]], *kind[1:], A, B, scale_a, scale_b, offsets, order, top_k, bias, out)
        if got is not None:
            return got
    name, fmt, per_byte, part, b_rows = kind
    dtypes = (torch.int8,) if b_rows == 0 else _E4M3 if per_byte == 1 else (torch.uint8,)
    sdtypes = _UE8M0 if fmt >= 0 else _F32
    (a_rows, row), lda = _rows(A, "A", dtypes)
    device = A.device
    if not isinstance(B, torch.Tensor) or B.dtype not in dtypes or B.device != device or B.dim() != 3:
        raise ValueError(f"B must be a tensor of {dtypes} [experts, N, K] on {device}")
    experts, N, brow = B.shape
    sb, ldb = B.stride(), B.stride(1) if N > 1 else brow
    if brow != row:
        raise ValueError(f"A has rows of {row} bytes, B of {brow}")
    if (brow > 1 and sb[2] != 1) or (experts > 1 and N > 0 and sb[0] != N * ldb):
        raise ValueError("B must have unit stride along K and its experts N rows apart")
    K = row * per_byte
    if not isinstance(offsets, torch.Tensor) or offsets.numel() != experts + 1:
        raise ValueError(f"offsets must hold {experts + 1} values")
    po = _vec(offsets, "offsets", experts + 1, device, (_I32,))
    if order is None:
        rows, pr, top_k = a_rows, None, 1
    else:
        if not isinstance(order, torch.Tensor) or order.dim() != 1:
            raise ValueError("order must be a 1-D tensor")
        rows = order.shape[0]
        pr = _vec(order, "order", rows, device, (_I32,))
        if top_k is None:
            if rows % max(a_rows, 1):
                raise ValueError(f"an order of {rows} slots for {a_rows} tokens: top_k has to be given")
            top_k = rows // a_rows if a_rows and rows else 1
        top_k = _count(top_k, "top_k", 64)
    psa = _table(scale_a, "scale_a", (a_rows, K // part) if part else (a_rows,), sdtypes, device)
    psb = _table(scale_b, "scale_b", (experts, -(-N // b_rows), K // part) if part else (experts, N), sdtypes, device)
    pb = None if bias is None else _table(bias, "bias", (experts, N), _BF16, device)
    if out is None:
        wide = N + (-N) % 8                   # the library's rule for row strides
        out, ldc = _new((rows, wide), torch.bfloat16, device, stream), wide
        out = out if wide == N else out[:, :N]
    else:
        out, ldc = _out_rows(out, "out", (rows, N), device, stream)
        ldc = ldc if rows > 1 else N + (-N) % 8
    _enqueue(getattr(L, name), device, stream, *((fmt,) if fmt >= 0 else ()), A.data_ptr(),
             lda if a_rows > 1 else row, a_rows, B.data_ptr(), ldb, psa, psb, po, pr, top_k, pb, out.data_ptr(), ldc,
             rows, experts, N, K)
    return out


def qgemm_i8_rowwise_grouped(A, B, scale_a, scale_b, offsets, order=None, top_k=None, bias=None, out=None, stream=None):
    """One qgemm_i8_rowwise per expert over its rows: rows offsets[e] ..
    offsets[e+1]-1 of the result are rows of A times B[e].  With an order (of
    the sort) A holds the tokens and row r takes token order[r] // top_k (None: as
    many slots a token as the order has for A's rows); without one A holds the
    rows.  A int8 [rows of A, K], B int8 [experts, N, K], scale_a fp32 [rows of A],
    scale_b fp32 [experts, N], bias bf16 [experts, N] -> bf16 [rows, N]; rows past
    offsets[experts] are left as they are.  K a multiple of 128."""
    return _grouped(_G_I8, A, B, scale_a, scale_b, offsets, order, top_k, bias, out, stream)


def qgemm_f8_pertoken_grouped(A, B, scale_a, scale_b, offsets, order=None, top_k=None, bias=None, out=None, stream=None):
    """One qgemm_f8_pertoken per expert over its rows; A, B e4m3 (uint8 or
    float8_e4m3fn), otherwise as qgemm_i8_rowwise_grouped."""
    return _grouped(_G_F8, A, B, scale_a, scale_b, offsets, order, top_k, bias, out, stream)


def qgemm_f8_blockscale_grouped(A, B, scale_a, scale_b, offsets, order=None, top_k=None, bias=None, out=None,
                                stream=None):
    """One qgemm_f8_blockscale per expert over its rows; scale_a fp32
    [rows of A, K/128], scale_b fp32 [experts, ceil(N/128), K/128], otherwise as
    qgemm_f8_pertoken_grouped."""
    return _grouped(_G_BLOCK, A, B, scale_a, scale_b, offsets, order, top_k, bias, out, stream)


def qgemm_mx_grouped(fmt, A, B, scale_a, scale_b, offsets, order=None, top_k=None, bias=None, out=None, stream=None):
    """One qgemm_mx per expert over its rows; A, B e4m3 or e2m1 (two codes a
    byte, rows of K/2 bytes), scale_a ue8m0 [rows of A, K/32], scale_b ue8m0
    [experts, N, K/32], otherwise as qgemm_i8_rowwise_grouped."""
    if fmt not in (QGEMM_MX_E4M3, QGEMM_MX_E2M1):
        raise ValueError(f"unknown MX format {fmt}")
    return _grouped(_G_MX[fmt], A, B, scale_a, scale_b, offsets, order, top_k, bias, out, stream)
