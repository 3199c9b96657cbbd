"""Plain CPU implementations of the 8-bit cache operators for the tests: the
append in IEEE binary32 steps (bit-exact), the attention in binary64 with the
bound that the kernel's roundings allow."""
import numpy as np
import torch

QMAX = {"e4m3": np.float32(448.0), "i8": np.float32(127.0)}
DTYPE = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def values(codes):
    """Codes (CPU tensor) as float64."""
    return codes.float().double().numpy() if codes.dtype != torch.int8 else codes.numpy().astype(np.float64)


def encode(v, fmt):
    """float32 array -> codes (uint8 view), nearest even, saturating."""
    if fmt == "i8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
    t = torch.from_numpy(np.clip(v, -448.0, 448.0).astype(np.float32))
    return t.to(torch.float8_e4m3fn).view(torch.uint8).numpy()


def append(cache, new_k, new_v, table, cu, lens, fmt):
    """cache: dict of CPU tensors k, v, k_scale, v_scale (changed in place);
    new_k, new_v CPU bf16 [tokens, heads, dim]."""
    blocks, heads, bs, _ = cache["k"].shape
    for name, x in (("k", new_k), ("v", new_v)):
        x = x.float().numpy()
        codes, scales = cache[name].view(torch.uint8).numpy(), cache[name + "_scale"].numpy()
        if name == "v":
            codes = codes.swapaxes(2, 3)
        for b, n in enumerate(lens):
            q = cu[b + 1] - cu[b]
            start = n - q
            for j in range(max(start, 0) // bs, -(-max(n, 0) // bs)):
                lo, hi = max(start, j * bs), min(n, (j + 1) * bs)
                if lo >= hi or j >= len(table[b]) or not 0 <= table[b][j] < blocks:
                    continue
                blk = table[b][j]
                for h in range(heads):
                    part = x[cu[b] + lo - start:cu[b] + hi - start, h]
                    was = scales[blk, h] if lo > j * bs else np.float32(0)
                    now = max(was, np.abs(part).max() * (np.float32(1) / QMAX[fmt]))
                    unit = now if now > 0 else np.float32(1)
                    old = codes[blk, h, :lo - j * bs]
                    if lo > j * bs and now > was:
                        v = torch.from_numpy(old.copy()).view(DTYPE[fmt]).float().numpy()
                        old[:] = encode((v * was) / unit, fmt)
                    codes[blk, h, lo - j * bs:hi - j * bs] = encode(part / unit, fmt)
                    scales[blk, h] = now


def attention(cache, Q, table, cu, lens, fmt, causal=True, window=0, sm_scale=None):
    """(float64 result [tokens, heads, dim], allowed absolute error).  The error:
    bf16 of the result (8 significant bits: 2^-8 |o| at most); binary16 of each
    weight (11 bits: 2^-11); binary32 sums of the scores over dim terms, which
    move a probability by the same relative amount, twice over (numerator and
    denominator); exp2 and the sums over tokens (2^-18 covers both)."""
    heads, dim = Q.shape[1], Q.shape[2]
    blocks, kvh, bs, _ = cache["k"].shape
    sm = dim ** -0.5 if sm_scale is None else sm_scale
    q64 = Q.float().double().numpy()
    out, tol = np.zeros(q64.shape), np.zeros(q64.shape)
    g = heads // kvh
    for b, n in enumerate(lens):
        nq = cu[b + 1] - cu[b]
        if n <= 0 or nq <= 0:
            continue
        here = [j for j in range(-(-n // bs)) if j < len(table[b]) and 0 <= table[b][j] < blocks]
        pos = np.concatenate([np.arange(j * bs, min((j + 1) * bs, n)) for j in here]) if here else np.zeros(0, int)
        for h in range(kvh):
            if not here:
                continue
            k = np.concatenate([values(cache["k"][table[b][j], h])[:min(bs, n - j * bs)]
                                * float(cache["k_scale"][table[b][j], h]) for j in here])
            v = np.concatenate([values(cache["v"][table[b][j], h]).T[:min(bs, n - j * bs)]
                                * float(cache["v_scale"][table[b][j], h]) for j in here])
            qq = q64[cu[b]:cu[b + 1], h * g:(h + 1) * g]                 # [nq, g, dim]
            at = n - nq + np.arange(nq)[:, None]
            seen = np.ones((nq, len(pos)), bool)
            if causal:
                seen = pos[None] <= at
                if window:
                    seen &= pos[None] > at - window
            for r in range(g):
                # codes that no row sees may be anything: leave them out before the products
                any_ = seen.any(0)
                if not any_.any():
                    continue
                kk, vv, se = k[any_], v[any_], seen[:, any_]
                s = np.where(se, qq[:, r] @ kk.T * sm, -np.inf)
                size = np.where(se, np.abs(qq[:, r]) @ np.abs(kk).T * abs(sm), 0).max(1, keepdims=True)
                top = s.max(1, keepdims=True)
                p = np.exp(s - np.where(np.isfinite(top), top, 0))
                tot = p.sum(1, keepdims=True)
                p = np.where(tot > 0, p / np.where(tot > 0, tot, 1), 0)
                o = p @ vv
                out[cu[b]:cu[b + 1], h * g + r] = o
                moved = 2 * (dim + 8) * 2.0 ** -24 * size
                tol[cu[b]:cu[b + 1], h * g + r] = (2.0 ** -8 * np.abs(o)
                                                   + (2.0 ** -11 + moved + 2.0 ** -18) * (p @ np.abs(vv)) + 2.0 ** -133)
    return out, tol
