"""The operators of a layer of experts around the grouped scaled GEMMs: cases,
plain forms and the definitions in 64 bits.

    sort       the (token, expert) choices of a router in order of experts
    exchange   tokens copied into that order and the experts' outputs summed
               back with weights, or the gradients of both
    experts    one scaled low-precision product per expert over its rows
    swiglu     silu(gate) * up between the experts' two products, output in 8
               bits with the scales of the product that follows
    postnorm   the norm after a block, its gate and residual scale, and the norm
               before the next block with output in 8 bits

``run`` computes them from elementary torch operations in float32 where
``own`` is false, and through the library where it is true.
"""
import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 64 sequences, 8 of 256 experts each: the latency of the sort
        {"name": "sort-decode", "op": "sort", "tokens": 64, "k": 8, "experts": 256, "ranks": 1},
        # a long prefill batch, an odd number of tokens
        {"name": "sort-prompt", "op": "sort", "tokens": 32769, "k": 8, "experts": 128, "ranks": 1},
        # the same decode step's rows to the experts and back onto the residual stream
        {"name": "exchange-decode", "op": "exchange", "tokens": 64, "k": 8, "experts": 256, "ranks": 1, "H": 7168,
         "residual": True, "grad": False},
        # a prompt's rows to the experts and back
        {"name": "exchange-prompt", "op": "exchange", "tokens": 8192, "k": 8, "experts": 64, "ranks": 1, "H": 7168,
         "residual": True, "grad": False},
        # the gradients of a training step on one of two ranks: half of the choices are the other's
        {"name": "exchange-grad", "op": "exchange", "tokens": 4095, "k": 6, "experts": 32, "ranks": 2, "H": 5376,
         "residual": False, "grad": True},
        # 16 tokens of a decode step through MXFP4 experts: one row for most of them, weights streamed
        {"name": "experts-decode", "op": "experts", "kind": "mx_e2m1", "tokens": 16, "k": 8, "experts": 128,
         "ranks": 1, "N": 4096, "K": 7168, "gather": True, "bias": False},
        # a short prompt through the second product of FP8 experts, rows already in their order
        {"name": "experts-mid", "op": "experts", "kind": "f8_block", "tokens": 1000, "k": 6, "experts": 64,
         "ranks": 1, "N": 7168, "K": 2048, "gather": False, "bias": False},
        # a prompt through the first product of INT8 experts, rows taken where the tokens lie
        {"name": "experts-prompt", "op": "experts", "kind": "i8", "tokens": 8192, "k": 4, "experts": 32,
         "ranks": 1, "N": 4096, "K": 7168, "gather": True, "bias": True},
        # between the products of a decode step
        {"name": "swiglu-decode", "op": "swiglu", "kind": "f8_pertoken", "M": 512, "I": 2048, "live": 512},
        # between the products of a prompt: room for more rows than came
        {"name": "swiglu-prompt", "op": "swiglu", "kind": "mx_e4m3", "M": 32768, "I": 2112, "live": 30001},
        # one token between two blocks
        {"name": "postnorm-token", "op": "postnorm", "kind": "f8_pertoken", "M": 1, "K": 7168, "gate": False,
         "alpha": 1.0},
        # a prompt between two blocks, with a gate for each channel and a residual scale
        {"name": "postnorm-prompt", "op": "postnorm", "kind": "f8_block", "M": 8191, "K": 5376, "gate": True,
         "alpha": 0.25},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 5e12, w["flops"] / 1e14)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["sort", "exchange", "exchange", "experts", "experts", "swiglu", "postnorm"])
        if op in ("sort", "exchange", "experts"):
            c = {"op": op, "k": rng.choice([1, 2, 4, 6, 8]), "experts": _log(rng, 8, 512 if op == "sort" else 128),
                 "ranks": rng.choice([1, 1, 2, 4])}
        if op == "sort":
            c["tokens"] = _log(rng, 1, 40000)
        elif op == "exchange":
            c.update(tokens=_log(rng, 1, 16384), H=8 * _log(rng, 128, 1024), residual=rng.random() < 0.5,
                     grad=rng.random() < 0.5)
            if c["tokens"] * c["k"] * c["H"] > 5e8:
                continue
        elif op == "experts":
            c.update(kind=rng.choice(["i8", "f8_pertoken", "f8_block", "mx_e2m1", "mx_e4m3"]),
                     tokens=_log(rng, 1, 8192), N=_log(rng, 128, 8192), K=128 * _log(rng, 8, 56),
                     gather=rng.random() < 0.5, bias=rng.random() < 0.3)
            if c["experts"] * c["N"] * c["K"] > 4e9:       # the weights in bytes
                continue
        elif op == "swiglu":
            c = {"op": op, "kind": rng.choice(["f8_pertoken", "f8_block", "mx_e4m3"]), "M": _log(rng, 1, 40000),
                 "I": 128 * _log(rng, 4, 64)}
            c["live"] = c["M"] if rng.random() < 0.5 else rng.randint(0, c["M"])
        else:
            c = {"op": op, "kind": rng.choice(["f8_pertoken", "f8_block", "mx_e4m3"]), "M": _log(rng, 1, 16384),
                 "K": 128 * _log(rng, 8, 100), "gate": rng.random() < 0.5, "alpha": rng.choice([1.0, 0.5, 0.22])}
        if _cost(c) <= most:
            return c


def _live(c):
    """Expected choices that fall on this rank's experts, and its experts that
    have any."""
    rows = c["tokens"] * c["k"] / c["ranks"]
    e = c["experts"]
    return rows, e * (1.0 - (1.0 - 1.0 / e) ** rows)


def work(case):
    c = case
    if c["op"] == "sort":
        s = c["tokens"] * c["k"]
        return {"bytes": 12 * s + 4 * c["experts"] + 4, "flops": s}
    if c["op"] == "exchange":
        rows, t, h = int(_live(c)[0]), c["tokens"], c["H"]
        if c["grad"]:
            # dout and y to dy and dw; dxs to dx
            return {"bytes": 2 * h * (t + 2 * rows) + 12 * t * c["k"] + 2 * h * (rows + t), "flops": 4 * rows * h}
        return {"bytes": 2 * h * (t + rows) + 2 * h * (rows + t * (2 if c["residual"] else 1)) + 12 * t * c["k"],
                "flops": 2 * rows * h}
    if c["op"] == "experts":
        rows, full = _live(c)
        n, k = c["N"], c["K"]
        b = {"mx_e2m1": k // 2 + k // 32, "mx_e4m3": k + k // 32, "f8_block": k + k // 4096, "i8": k,
             "f8_pertoken": k}[c["kind"]]
        a = (k // 2 if c["kind"] == "mx_e2m1" else k) + (k // 32 if c["kind"] not in ("i8", "f8_pertoken") else 4)
        a_rows = min(rows, c["tokens"]) if c["gather"] else rows
        return {"bytes": int(full * n * b + a_rows * a + 2 * rows * n), "flops": int(2 * rows * n * k)}
    if c["op"] == "swiglu":
        n = c["live"] * c["I"]
        return {"bytes": 5 * n + (n // 32 if c["kind"] != "f8_pertoken" else 4 * c["live"]), "flops": 8 * n}
    n = c["M"] * c["K"]
    return {"bytes": 7 * n + (6 if c["gate"] else 4) * c["K"] + (n // 32 if c["kind"] != "f8_pertoken" else 4 * c["M"]),
            "flops": 16 * n}


# ---------------------------------------------------------------- inputs

def _route(c, gen):
    """A router's choices for each token: k different ones of all ranks'
    experts, some experts chosen more often; this rank's are 0 .. experts - 1."""
    total = c["experts"] * c["ranks"]
    bias = torch.randn(total, device=DEV, generator=gen) * 0.5
    logits = torch.randn(c["tokens"], total, device=DEV, generator=gen) + bias
    top, ids = logits.topk(min(c["k"], total), dim=1)
    first = c["experts"] * (c["ranks"] // 2)
    return (ids - first).int().contiguous(), torch.softmax(top, 1)


def _sorted(ids, experts):
    """(offsets, order, position) of the choices, as the sort leaves them."""
    flat = ids.reshape(-1).long()
    slots = flat.numel()
    key = torch.where((flat >= 0) & (flat < experts), flat, experts)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=DEV)).int()
    at = torch.arange(slots, device=DEV)
    live = at < offsets[-1]
    position = torch.empty(slots, dtype=torch.int32, device=DEV)
    position[order] = torch.where(live, at, -1).int()
    return offsets, torch.where(live, order, -1).int(), position.view(ids.shape)


def _e4m3(shape, gen):
    """Codes as a quantiser leaves them for normal data whose largest of a
    block is about four deviations."""
    out = torch.empty(shape, dtype=torch.float8_e4m3fn, device=DEV)
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        x = torch.randn(min(1 << 27, flat.numel() - at), device=DEV, generator=gen)
        flat[at:at + x.numel()] = x.mul_(112.0).clamp_(-448.0, 448.0).to(out.dtype)
    return out


def _bytes(shape, gen, lo=0, hi=256, dtype=torch.uint8):
    return torch.randint(lo, hi, shape, dtype=dtype, device=DEV, generator=gen)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device=DEV, generator=gen)

    def bf16(*shape):
        return torch.randn(*shape, device=DEV, generator=gen, dtype=torch.bfloat16)

    if c["op"] == "swiglu":
        x = bf16(c["M"], 2 * c["I"])
        s = {"case": c, "x": x, "count": torch.tensor([c["live"]], dtype=torch.int32, device=DEV)}
        parts = {"f8_pertoken": 1, "f8_block": c["I"] // 128, "mx_e4m3": c["I"] // 32}[c["kind"]]
        s["codes"] = torch.zeros(c["M"], c["I"], dtype=torch.uint8, device=DEV)   # rows behind the last stay zero
        s["scale"] = torch.zeros((c["M"], parts) if parts > 1 else (c["M"],), device=DEV,
                                 dtype=torch.uint8 if c["kind"] == "mx_e4m3" else torch.float32)
        return s
    if c["op"] == "postnorm":
        r = normal(c["M"], c["K"])
        r[:, 5::97] *= 20.0                           # channels that stand out, as in a residual stream
        return {"case": c, "y": (normal(c["M"], c["K"]) * 3.0).bfloat16(), "residual": r.bfloat16(),
                "gamma_post": (1.0 + 0.1 * normal(c["K"])).bfloat16(),
                "gamma": (1.0 + 0.1 * normal(c["K"])).bfloat16(),
                "gate": torch.tanh(normal(c["K"])).bfloat16() if c["gate"] else None}
    ids, weights = _route(c, gen)
    s = {"case": c, "ids": ids}
    if c["op"] == "sort":
        return s
    s["offsets"], s["order"], s["position"] = _sorted(ids, c["experts"])
    rows, t = ids.numel(), c["tokens"]
    if c["op"] == "exchange":
        h = c["H"]
        s["weights"] = weights.contiguous()
        s["y"] = bf16(rows, h)
        if c["grad"]:
            s["dout"], s["dxs"] = bf16(t, h), bf16(rows, h)
        else:
            s["x"] = bf16(t, h)
            s["residual"] = bf16(t, h) if c["residual"] else None
        s["rows"] = torch.zeros(rows, h, dtype=torch.bfloat16, device=DEV)       # xs or dy; rows without expert stay
        return s
    n, k, e = c["N"], c["K"], c["experts"]
    m = t if c["gather"] else rows
    # counts on the host, for the plain form's loop over experts
    s["counts"] = (s["offsets"][1:] - s["offsets"][:-1]).tolist()
    if c["kind"] == "i8":
        s["a"] = normal(m, k).mul_(31.75).round_().clamp_(-127.0, 127.0).to(torch.int8)
        s["b"] = _bytes((e, n, k), gen, -127, 128, torch.int8)
        s["sa"] = 1e-3 + 9e-3 * torch.rand(m, device=DEV, generator=gen)
        s["sb"] = 1e-3 + 9e-3 * torch.rand(e, n, device=DEV, generator=gen)
    elif c["kind"] in ("f8_pertoken", "f8_block"):
        s["a"], s["b"] = _e4m3((m, k), gen), _e4m3((e, n, k), gen)
        block = c["kind"] == "f8_block"
        s["sa"] = (3.0 + 2.0 * torch.rand((m, k // 128) if block else (m,), device=DEV, generator=gen)) / 448.0
        s["sb"] = (0.05 + 0.05 * torch.rand((e, -(-n // 128), k // 128) if block else (e, n), device=DEV,
                                            generator=gen)) / 448.0
    else:
        if c["kind"] == "mx_e4m3":
            s["a"], s["b"] = _e4m3((m, k), gen), _e4m3((e, n, k), gen)
        else:
            s["a"], s["b"] = _bytes((m, k // 2), gen), _bytes((e, n, k // 2), gen)
        s["sa"], s["sb"] = _bytes((m, k // 32), gen, 119, 122), _bytes((e, n, k // 32), gen, 117, 122)
    s["bias"] = bf16(e, n) if c["bias"] else None
    s["out"] = torch.zeros(rows, n + (-n) % 8, dtype=torch.bfloat16, device=DEV)[:, :n]   # rows without expert stay
    return s


# ---------------------------------------------------------------- the passes

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"sort": _sort, "exchange": _exchange, "experts": _experts, "swiglu": _swiglu,
                "postnorm": _postnorm}[c["op"]](s, c)
    import block_scaled_precision_02_amd as lib
    if c["op"] == "sort":
        offsets, order, position = lib.qgemm_moe_sort(s["ids"], c["experts"])
        return {"offsets": offsets, "order": order, "position": position}
    if c["op"] == "exchange":
        if c["grad"]:
            dy, dw = lib.qgemm_moe_combine_grad(s["dout"], s["y"], s["position"], s["weights"], dY=s["rows"])
            return {"dy": dy, "dweights": dw, "dx": lib.qgemm_moe_combine(s["dxs"], s["position"])}
        xs = lib.qgemm_moe_gather(s["x"], s["position"], out=s["rows"])
        out = lib.qgemm_moe_combine(s["y"], s["position"], s["weights"], residual=s["residual"])
        return {"xs": xs, "out": out}
    if c["op"] == "experts":
        args = dict(order=s["order"], top_k=c["k"]) if c["gather"] else {}
        args.update(bias=s["bias"], out=s["out"])
        if c["kind"] in ("mx_e2m1", "mx_e4m3"):
            fmt = lib.QGEMM_MX_E2M1 if c["kind"] == "mx_e2m1" else lib.QGEMM_MX_E4M3
            return lib.qgemm_mx_grouped(fmt, s["a"], s["b"], s["sa"], s["sb"], s["offsets"], **args)
        f = {"i8": lib.qgemm_i8_rowwise_grouped, "f8_pertoken": lib.qgemm_f8_pertoken_grouped,
             "f8_block": lib.qgemm_f8_blockscale_grouped}[c["kind"]]
        return f(s["a"], s["b"], s["sa"], s["sb"], s["offsets"], **args)
    if c["op"] == "swiglu":
        args = dict(count=s["count"], out=s["codes"], scale=s["scale"])
        if c["kind"] == "mx_e4m3":
            codes, scale = lib.qgemm_swiglu_quant_mx(lib.QGEMM_MX_E4M3, s["x"], **args)
        else:
            f = lib.qgemm_swiglu_quant_f8_pertoken if c["kind"] == "f8_pertoken" else lib.qgemm_swiglu_quant_f8_block
            codes, scale = f(s["x"], **args)
        return _coded(codes, scale)
    args = (s["y"], s["residual"], s["gamma_post"], s["gamma"], EPS)
    kw = dict(gate=s["gate"], alpha=c["alpha"])
    if c["kind"] == "mx_e4m3":
        codes, scale, out = lib.qgemm_postnorm_quant_mx(lib.QGEMM_MX_E4M3, *args, **kw)
    else:
        f = lib.qgemm_postnorm_quant_f8_pertoken if c["kind"] == "f8_pertoken" else lib.qgemm_postnorm_quant_f8_block
        codes, scale, out = f(*args, **kw)
    return dict(_coded(codes, scale), residual=out)


def _coded(codes, scale):
    return {"codes": codes.view(torch.float8_e4m3fn),
            "scale": scale.view(torch.float8_e8m0fnu) if scale.dtype == torch.uint8 else scale}


def _sort(s, c):
    offsets, order, position = _sorted(s["ids"], c["experts"])
    return {"offsets": offsets, "order": order, "position": position}


def _back(y, position, weights, base):
    """base + the sum over a token's choices of weight times row."""
    acc = base
    for j in range(position.shape[1]):
        p = position[:, j].long()
        w = (p >= 0).float() if weights is None else torch.where(p >= 0, weights[:, j], 0.0)
        acc = acc + w[:, None] * y[p.clamp(min=0)].float()
    return acc.bfloat16()


def _exchange(s, c):
    t, h, k = c["tokens"], c["H"], s["position"].shape[1]
    order = s["order"].long()
    live = (order >= 0)[:, None]
    token = order.clamp(min=0) // k
    if not c["grad"]:
        xs = torch.where(live, s["x"][token], 0.0)
        base = s["residual"].float() if c["residual"] else torch.zeros(t, h, device=DEV)
        return {"xs": xs, "out": _back(s["y"], s["position"], s["weights"], base)}
    w = s["weights"].reshape(-1)[order.clamp(min=0)][:, None]
    dout = s["dout"].float()
    dy = torch.where(live, w * dout[token], 0.0).bfloat16()
    dw = torch.stack([torch.where(p >= 0, (dout * s["y"][p.clamp(min=0).long()].float()).sum(1), 0.0)
                      for p in s["position"].unbind(1)], 1)
    return {"dy": dy, "dweights": dw, "dx": _back(s["dxs"], s["position"], None, torch.zeros(t, h, device=DEV))}


_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _values(codes, scale, kind, k):
    """The float32 values of rows of codes (without per-row scales)."""
    if kind in ("i8", "f8_pertoken"):
        return codes.float()
    if kind == "mx_e2m1":
        v = torch.tensor(_E2M1, device=DEV)[torch.stack((codes & 15, codes >> 4), 2).int()].view(-1, k // 32, 32)
    else:
        v = codes.float().view(-1, k // (128 if kind == "f8_block" else 32), 128 if kind == "f8_block" else 32)
    unit = scale if kind == "f8_block" else torch.exp2(scale.float() - 127.0)
    return (v * unit[..., None]).view(-1, k)


def _experts(s, c):
    k, n, kind = c["K"], c["N"], c["kind"]
    out, at = s["out"], 0
    for e, count in enumerate(s["counts"]):
        if count == 0:
            continue
        rows = torch.arange(at, at + count, device=DEV)
        if c["gather"]:
            rows = s["order"][at:at + count].long() // s["ids"].shape[1]
        sa, sb = s["sa"][rows], s["sb"][e]
        codes = s["a"][rows] if c["kind"] in ("i8", "mx_e2m1") else s["a"].view(torch.uint8)[rows].view(s["a"].dtype)
        a = _values(codes, sa, kind, k)
        b = _values(s["b"][e], sb.repeat_interleave(128, 0)[:n] if kind == "f8_block" else sb, kind, k)
        y = a @ b.t()
        if kind in ("i8", "f8_pertoken"):
            y = y * sa[:, None] * sb[None, :]
        if s["bias"] is not None:
            y = y + s["bias"][e].float()
        out[at:at + count] = y.bfloat16()
        at += count
    return out


def _quantised(y, kind):
    """Codes and scales of float32 rows."""
    m, k = y.shape
    if kind == "mx_e4m3":
        b = y.view(m, k // 32, 32)
        e = torch.frexp(b.abs().amax(2, keepdim=True))[1] - 1          # floor(log2 amax)
        code = (e - 8 + 127).clamp(0, 254)
        v = torch.ldexp(b, 127 - code).clamp(-448.0, 448.0)
        scale = code.squeeze(2).to(torch.uint8).view(torch.float8_e8m0fnu)
    else:
        b = y.view(m, -1, 128 if kind == "f8_block" else k)
        scale = b.abs().amax(2, keepdim=True) / 448.0
        v = b / torch.where(scale > 0, scale, 1.0)
        scale = scale.view(m) if kind == "f8_pertoken" else scale.squeeze(2)
    return {"codes": v.reshape(m, k).to(torch.float8_e4m3fn), "scale": scale}


def _swiglu(s, c):
    g, u = s["x"][:, :c["I"]].float(), s["x"][:, c["I"]:].float()
    got = _quantised(g / (1.0 + torch.exp(-g)) * u, c["kind"])
    live = (torch.arange(c["M"], device=DEV) < s["count"])[:, None]
    codes = torch.where(live, got["codes"].view(torch.uint8), 0)
    scale = got["scale"]
    if scale.dim() == 1:
        scale = torch.where(live[:, 0], scale, 0.0)
    elif scale.dtype == torch.float32:
        scale = torch.where(live, scale, 0.0)
    else:
        scale = torch.where(live, scale.view(torch.uint8), 0).view(scale.dtype)
    return {"codes": codes.view(torch.float8_e4m3fn), "scale": scale}


def _postnorm(s, c):
    y = s["y"].float()
    n = y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["gamma_post"].float()
    if s["gate"] is not None:
        n = n * s["gate"].float()
    h = s["residual"].float() + c["alpha"] * n
    z = h * torch.rsqrt((h * h).mean(1, keepdim=True) + EPS) * s["gamma"].float()
    return dict(_quantised(z, c["kind"]), residual=h.bfloat16())


# ---------------------------------------------------------------- definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    return {"sort": _exact_sort, "exchange": _exact_exchange, "experts": _exact_experts, "swiglu": _exact_swiglu,
            "postnorm": _exact_postnorm}[c["op"]](s, c)


def _exact_sort(s, c):
    ids = s["ids"].cpu().numpy().astype(np.int64)
    flat = ids.reshape(-1)
    lists = [np.flatnonzero(flat == e) for e in range(c["experts"])]
    offsets = np.cumsum([0] + [len(x) for x in lists])
    order = np.full(flat.size, -1, np.int64)
    position = np.full(flat.size, -1, np.int64)
    for at, x in zip(offsets, lists):
        order[at:at + len(x)] = x
        position[x] = at + np.arange(len(x))
    return {"offsets": torch.from_numpy(offsets).int().to(DEV), "order": torch.from_numpy(order).int().to(DEV),
            "position": torch.from_numpy(position.reshape(ids.shape)).int().to(DEV)}


def _exact_exchange(s, c):
    t, h = c["tokens"], c["H"]
    pos = s["position"].long()
    slot_token = torch.arange(t, device=DEV)[:, None].expand_as(pos)
    has = pos >= 0
    to, of = pos[has], slot_token[has]                    # row, token of every live choice
    if c["grad"]:
        w = s["weights"].double()[has]
        dy = torch.zeros(pos.numel(), h, dtype=torch.float64, device=DEV)
        dw = torch.zeros(pos.shape, dtype=torch.float64, device=DEV)
        dx = torch.zeros(t, h, dtype=torch.float64, device=DEV)
        dots = torch.empty(to.numel(), dtype=torch.float64, device=DEV)
        for a in range(0, to.numel(), 8192):
            z = slice(a, a + 8192)
            d = s["dout"][of[z]].double()
            dy[to[z]] = d * w[z, None]
            dots[z] = torch.einsum("rh,rh->r", d, s["y"][to[z]].double())
            dx.index_add_(0, of[z], s["dxs"][to[z]].double())
        dw[has] = dots
        return {"dy": dy, "dweights": dw, "dx": dx}
    out = s["residual"].double() if c["residual"] else torch.zeros(t, h, dtype=torch.float64, device=DEV)
    xs = torch.zeros(pos.numel(), h, dtype=torch.float64, device=DEV)
    w = s["weights"].double()[has]
    for a in range(0, to.numel(), 8192):
        z = slice(a, a + 8192)
        xs[to[z]] = s["x"][of[z]].double()
        out.index_add_(0, of[z], s["y"][to[z]].double() * w[z, None])
    return {"xs": xs, "out": out}


def _exact_experts(s, c):
    k, n, kind = c["K"], c["N"], c["kind"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist()
    table = torch.tensor(_E2M1, dtype=torch.float64, device=DEV)

    def wide(codes, scales, rows_per_scale):
        if kind in ("i8", "f8_pertoken"):
            return codes.double() * scales.double()[:, None]
        if kind == "mx_e2m1":
            v = torch.empty(codes.shape[0], k, dtype=torch.float64, device=DEV)
            v[:, 0::2], v[:, 1::2] = table[(codes & 15).long()], table[(codes >> 4).long()]
        else:
            v = codes.double()
        unit = scales.double() if kind == "f8_block" else 2.0 ** (scales.double() - 127)
        unit = unit[torch.arange(codes.shape[0], device=DEV) // rows_per_scale]
        return v * unit.repeat_interleave(128 if kind == "f8_block" else 32, 1)

    for e in range(c["experts"]):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        rows = s["order"][lo:hi].long() // s["ids"].shape[1] if c["gather"] else torch.arange(lo, hi, device=DEV)
        codes = s["a"].view(torch.uint8)[rows].view(s["a"].dtype)
        y = torch.mm(wide(codes, s["sa"][rows], 1),
                     wide(s["b"][e], s["sb"][e], 128 if kind == "f8_block" else 1).t().contiguous())
        if s["bias"] is not None:
            y += s["bias"][e].double()
        out[lo:hi] = y
    return out


def _enc(v):
    """The e4m3 values nearest to v (float64), ties to even."""
    v = v.clamp(-448, 448)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_codes(y, kind):
    parts = {"f8_pertoken": 1, "f8_block": y.shape[1] // 128, "mx_e4m3": y.shape[1] // 32}[kind]
    b = y.view(y.shape[0], parts, -1)
    top = b.abs().amax(2, keepdim=True)
    sc = torch.exp2(torch.floor(torch.log2(top)) - 8) if kind == "mx_e4m3" else top / 448
    return _enc(b / sc).view(y.shape), sc.squeeze(2)


def _exact_swiglu(s, c):
    codes = torch.zeros(c["M"], c["I"], dtype=torch.float64, device=DEV)
    scale = torch.zeros(s["scale"].shape, dtype=torch.float64, device=DEV)
    if c["kind"] == "mx_e4m3":
        scale.fill_(2.0 ** -127)                       # what a scale byte of zero stands for
    for r in range(0, c["live"], 4096):
        z = slice(r, min(r + 4096, c["live"]))
        g, u = s["x"][z].double().chunk(2, 1)
        codes[z], sc = _exact_codes(g * torch.sigmoid(g) * u, c["kind"])
        scale[z] = sc.squeeze(1) if c["kind"] == "f8_pertoken" else sc
    return {"codes": codes, "scale": scale}


def _exact_postnorm(s, c):
    out = {"codes": [], "scale": [], "residual": []}
    for r in range(0, c["M"], 2048):
        y = s["y"][r:r + 2048].double()
        n = y / torch.sqrt(y.pow(2).sum(1, keepdim=True) / c["K"] + EPS) * s["gamma_post"].double()
        if c["gate"]:
            n *= s["gate"].double()
        h = s["residual"][r:r + 2048].double().add(n, alpha=c["alpha"])
        z = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / c["K"] + EPS) * s["gamma"].double()
        codes, sc = _exact_codes(z, c["kind"])
        out["codes"].append(codes)
        out["scale"].append(sc.squeeze(1) if c["kind"] == "f8_pertoken" else sc)
        out["residual"].append(h)
    return {name: torch.cat(parts) for name, parts in out.items()}
