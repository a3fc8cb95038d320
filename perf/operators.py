"""Cases of the microscaled linear layer and the root-mean-square norm, for measurement.

run() computes a case in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, where `own` is true, by the calls that a
program makes of this package.  exact() gives the same outputs from the
operators' definitions in 64 bits.

The block format: 32 consecutive columns of a row share one power-of-two scale
(a byte s, 2^(s-127)) and hold e4m3 or e2m1 codes.  Rows of codes and scales
are padded with zero bytes to a multiple of 128 columns; e2m1 holds two codes
in a byte, the even column in the low half.
"""

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a decoder block's input norm, with the residual's addition
        {"name": "norm_one_token", "op": "norm", "rows": 1, "cols": 4096, "type": "f16", "mx": False},
        # a prompt's norm in front of a microscaled product: 8-bit output with block scales
        {"name": "norm_prompt_mx", "op": "norm", "rows": 2048, "cols": 4096, "type": "bf16", "mx": True},
        # fine-tuning: the norm's gradient over a batch of sequences, the residual's gradient joined
        {"name": "norm_grad_batch", "op": "norm_grad", "rows": 8192, "cols": 4096, "type": "bf16", "dh": True},
        # the same at a small width, with a row count that fills no tile
        {"name": "norm_grad_ragged", "op": "norm_grad", "rows": 333, "cols": 1000, "type": "f16", "dh": False},
        # a trained weight into 4 bits, and its values back for the error's evaluation
        {"name": "quantize_weight", "op": "quantize", "rows": 4096, "cols": 14336, "type": "f32", "fmt": "e2m1"},
        # activations of a mid-size batch whose width ends inside a block
        {"name": "quantize_ragged", "op": "quantize", "rows": 300, "cols": 257, "type": "f16", "fmt": "e4m3"},
        # one token through an MLP's up projection
        {"name": "linear_one_token", "op": "linear", "batch": 1, "n": 14336, "m": 4096, "type": "f16",
         "act": "e4m3", "ready": False},
        # sixteen sequences decoded together through the down projection
        {"name": "linear_decode_batch", "op": "linear", "batch": 16, "n": 4096, "m": 14336, "type": "bf16",
         "act": "e4m3", "ready": False},
        # a prompt through the up projection, activations quantised in the call
        {"name": "linear_prompt", "op": "linear", "batch": 2048, "n": 14336, "m": 4096, "type": "bf16",
         "act": "e4m3", "ready": False},
        # a prompt through the down projection, activations already in 4 bits
        {"name": "linear_prompt_fp4", "op": "linear", "batch": 2048, "n": 4096, "m": 14336, "type": "f16",
         "act": "e2m1", "ready": True},
        # fine-tuning through the frozen 4-bit weight: the input's gradient
        {"name": "linear_grad_prompt", "op": "linear_grad", "batch": 2048, "n": 14336, "m": 4096, "type": "bf16"},
        # the same at sizes that end inside blocks and tiles
        {"name": "linear_grad_ragged", "op": "linear_grad", "batch": 77, "n": 1000, "m": 1300, "type": "f16"},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm; half of them a multiple of 64 where that fits."""
    v = int(round(low * (high / low) ** rng.random()))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "quantize", "linear", "linear", "linear", "linear_grad"])
    t = rng.choice(["f16", "bf16"])
    if op in ("norm", "norm_grad"):
        c = {"op": op, "rows": _spread(rng, 1, 8192), "cols": _spread(rng, 32, 16384), "type": t}
        while c["rows"] * c["cols"] > 8192 * 4096:
            c["rows"] = max(1, c["rows"] // 2)
        c["mx" if op == "norm" else "dh"] = rng.random() < 0.5
        return c
    if op == "quantize":
        c = {"op": op, "rows": _spread(rng, 1, 14336), "cols": _spread(rng, 17, 14336),
             "type": rng.choice(["f16", "bf16", "f32"]), "fmt": rng.choice(["e4m3", "e2m1"])}
        while c["rows"] * c["cols"] > 4096 * 14336:
            c["rows"] = max(1, c["rows"] // 2)
        return c
    n, m = _spread(rng, 64, 14336), _spread(rng, 64, 14336)
    while n * m > 4096 * 14336:
        n = max(64, n // 2)
    c = {"op": op, "batch": _spread(rng, 1, 2048), "n": n, "m": m, "type": t}
    if op == "linear":
        c["act"] = rng.choice(["e4m3", "e2m1"])
        c["ready"] = rng.random() < 0.4
    return c


def work(case):
    if case["op"] == "norm":
        e = case["rows"] * case["cols"]
        return {"bytes": 6 * e + (e * 33 // 32 if case["mx"] else 2 * e) + 2 * case["cols"], "flops": 6 * e}
    if case["op"] == "norm_grad":
        e = case["rows"] * case["cols"]
        return {"bytes": (8 if case["dh"] else 6) * e + 4 * case["rows"] + 6 * case["cols"], "flops": 12 * e}
    if case["op"] == "quantize":
        e = case["rows"] * case["cols"]
        size = 4 if case["type"] == "f32" else 2
        # the 4-bit case also gives the values back in 16 bits
        return {"bytes": e * size + (e // 2 + e // 32 + 2 * e if case["fmt"] == "e2m1" else e + e // 32),
                "flops": 4 * e}
    b, n, m = case["batch"], case["n"], case["m"]
    weight = n * m // 2 + n * m // 32
    if case["op"] == "linear":
        size = 2 if not case["ready"] else 33 / 32 if case["act"] == "e4m3" else 17 / 32
        return {"bytes": weight + b * m * size + 2 * b * n, "flops": 2 * b * n * m}
    return {"bytes": weight + 2 * b * (n + m), "flops": 2 * b * n * m}


# ------------------------------------------------------- the block format, plain

# format: largest value's exponent, mantissa bits, smallest normal exponent, largest value
FORMATS = {"e4m3": (8, 3, -6, 448.0), "e2m1": (2, 1, 0, 6.0)}


def _blocks(x):
    """(rows, cols) in blocks of 32: (rows, blocks, 32), zeros after the last column."""
    rows, cols = x.shape
    return torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, -1, 32)


def _exponent(x):
    """floor(log2 |x|) of float32 values (normal ones; -127 and below for the rest)."""
    return ((x.view(torch.int32) >> 23) & 255) - 127


def _quantise(x, fmt):
    """(codes as the values they stand for, before the scale; scale bytes) of float32 (rows, cols)."""
    emax, mant, emin, top = FORMATS[fmt]
    b = _blocks(x)
    amax = b.abs().amax(dim=2)
    s = (_exponent(amax) - emax + 127).clamp(0, 254)
    bad = ~torch.isfinite(amax)
    s = torch.where(bad, 255, s)
    v = torch.ldexp(b, 127 - torch.where(bad, 127, s).unsqueeze(2))
    step = torch.ldexp(torch.ones_like(v), _exponent(v).clamp(min=emin) - mant)
    q = (torch.round(v / step) * step).clamp(-top, top)
    q = torch.where(bad.unsqueeze(2), 0.0, q)
    return q.reshape(x.shape[0], -1)[:, :x.shape[1]], s


def _scale(s):
    """float32 scales of scale bytes."""
    one = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.to(torch.int32) - 127)
    return torch.where(s == 255, float("nan"), one)


def _values(q, s):
    return q * _scale(s).repeat_interleave(32, dim=1)[:, :q.shape[1]]


def _pack(q, s, fmt):
    """Code values and scale bytes in the padded rows that a program holds."""
    rows, cols = q.shape
    wide = -(-cols // 128) * 128
    q = torch.nn.functional.pad(q, (0, wide - cols))
    s = torch.nn.functional.pad(s.to(torch.uint8), (0, wide // 32 - s.shape[1]))
    if fmt == "e4m3":
        return q.to(torch.float8_e4m3fn).view(torch.uint8).contiguous(), s.contiguous()
    a = q.abs()
    code = (2 * a).where(a <= 2, torch.where(a == 3, 5.0, torch.where(a == 4, 6.0, 7.0))).to(torch.uint8)
    code = code + 8 * (q < 0).to(torch.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous(), s.contiguous()


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _unpack(codes, scales, cols, fmt):
    """float32 values of packed rows."""
    if fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).to(torch.float32)
    else:
        table = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
        q = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), dim=2).reshape(codes.shape[0], -1)
    return _values(q, scales)[:, :cols]


# ------------------------------------------------------------------ the inputs

def _activations(gen, rows, cols, dtype):
    """Hidden states: normal, a few columns much larger than the rest, as residual streams have."""
    dev = gen.device
    x = torch.randn(rows, cols, generator=gen, device=dev)
    big = torch.rand(cols, generator=gen, device=dev) < 0.01
    return (x * torch.where(big, 12.0, 1.0)).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev, t, op = gen.device, TYPES[case["type"]], case["op"]
    st = {"case": case}
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        st["x"] = _activations(gen, rows, cols, t)
        st["residual"] = _activations(gen, rows, cols, t)
        st["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device=dev)).to(t)
    elif op == "norm_grad":
        rows, cols = case["rows"], case["cols"]
        st["h"] = _activations(gen, rows, cols, t)
        st["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device=dev)).to(t)
        st["dy"] = (0.01 * torch.randn(rows, cols, generator=gen, device=dev)).to(t)
        st["dh"] = (0.01 * torch.randn(rows, cols, generator=gen, device=dev)).to(t) if case["dh"] else None
        # kept from the forward pass
        st["rstd"] = torch.rsqrt(st["h"].float().square().mean(dim=1) + EPS)
    elif op == "quantize":
        rows, cols = case["rows"], case["cols"]
        if case["type"] == "f32":
            st["x"] = 0.02 * torch.randn(rows, cols, generator=gen, device=dev)
        else:
            st["x"] = _activations(gen, rows, cols, t)
    else:
        b, n, m = case["batch"], case["n"], case["m"]
        w = 0.02 * torch.randn(n, m, generator=gen, device=dev)
        st["codes"], st["scales"] = _pack(*_quantise(w, "e2m1"), "e2m1")
        del w
        if op == "linear_grad":
            st["dy"] = (0.01 * torch.randn(b, n, generator=gen, device=dev)).to(t)
        else:
            x = _activations(gen, b, m, t)
            if case["ready"]:
                st["xcodes"], st["xscales"] = _pack(*_quantise(x.float(), case["act"]), case["act"])
            else:
                st["x"] = x
        if own:
            import dbf_linear_fwd_amd as dbf
            st["layer"] = dbf.Layer.mx(dbf.MxTensor(st["codes"], st["scales"], m, "e2m1"), max_batch=b,
                                       act=case.get("act", "e4m3"))
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import dbf_linear_fwd_amd as dbf
    case = st["case"]
    op = case["op"]
    if op == "norm":
        r = dbf.rms_norm(st["x"], st["weight"], residual=st["residual"], eps=EPS, mx=case["mx"])
        if case["mx"]:
            return {"h": r.h, "y": _as_float8(r.y)}
        return {"h": r.h, "y": r.y}
    if op == "norm_grad":
        dx, dw = dbf.rms_norm_backward(st["dy"], st["h"], st["weight"], st["rstd"], dh=st["dh"])
        return {"dx": dx, "dweight": dw}
    if op == "quantize":
        q = dbf.mx_quantize(st["x"], case["fmt"])
        return _as_float8(q) if case["fmt"] == "e4m3" else {"values": q.dequantize(torch.bfloat16)}
    if op == "linear":
        x = dbf.MxTensor(st["xcodes"], st["xscales"], case["m"], case["act"]) if case["ready"] else st["x"]
        return {"y": st["layer"].forward(x, out_dtype=TYPES[case["type"]])}
    return {"dx": st["layer"].backward_data(st["dy"])}


def _as_float8(q):
    """A quantised tensor's bytes as the 8-bit floating types that torch has for them."""
    return {"codes": q.codes.view(torch.float8_e4m3fn)[:, :q.cols],
            "scales": q.scales.view(torch.float8_e8m0fnu)[:, :-(-q.cols // 32)]}


def _plain_float8(q, s):
    return {"codes": q.to(torch.float8_e4m3fn), "scales": s.to(torch.uint8).view(torch.float8_e8m0fnu)}


def _run_plain(st):
    case = st["case"]
    op, t = case["op"], TYPES[case["type"]]
    if op == "norm":
        h = (st["x"].float() + st["residual"].float()).to(t)
        # 64 bits: the values next to a rounding border of 8 bits
        hd = h.double()
        y = hd / torch.sqrt(hd.square().mean(dim=1, keepdim=True) + EPS) * st["weight"].double()
        if case["mx"]:
            return {"h": h, "y": _plain_float8(*_quantise(y.float(), "e4m3"))}
        return {"h": h, "y": y.float().to(t)}
    if op == "norm_grad":
        dy, h, w, rstd = st["dy"].float(), st["h"].float(), st["weight"].float(), st["rstd"].unsqueeze(1)
        g = dy * w
        dx = rstd * (g - h * (rstd * rstd * (g * h).mean(dim=1, keepdim=True)))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return {"dx": dx.to(t), "dweight": (dy * h * rstd).sum(dim=0)}
    if op == "quantize":
        q, s = _quantise(st["x"].float(), case["fmt"])
        return _plain_float8(q, s) if case["fmt"] == "e4m3" else {"values": _values(q, s).to(torch.bfloat16)}
    w = _unpack(st["codes"], st["scales"], case["m"], "e2m1")
    if op == "linear":
        if case["ready"]:
            x = _unpack(st["xcodes"], st["xscales"], case["m"], case["act"])
        else:
            x = _values(*_quantise(st["x"].float(), case["act"]))
        return {"y": (x @ w.t()).to(t)}
    return {"dx": (st["dy"].float() @ w).to(t)}


# ------------------------------------------------------------------ in 64 bits

def _positive_values(fmt):
    _, mant, emin, top = FORMATS[fmt]
    vals = [k * 2.0 ** (emin - mant) for k in range(2 ** mant)]
    e = emin
    while vals[-1] < top:
        vals += [v for v in ((2 ** mant + k) * 2.0 ** (e - mant) for k in range(2 ** mant)) if v <= top]
        e += 1
    return vals


def _nearest(v, fmt):
    """The format's value nearest to each of v (ties to the even code), by search among its values."""
    table = torch.tensor(_positive_values(fmt), dtype=torch.float64, device=v.device)
    mid = (table[1:] + table[:-1]) / 2
    a = v.abs()
    at = torch.bucketize(a, mid)
    tie = (at < mid.numel()) & (a == mid[at.clamp(max=mid.numel() - 1)])
    at = at + (tie & (at % 2 == 1)).to(at.dtype)
    return torch.copysign(table[at], v)


def _quantise64(x, fmt):
    """(code values, scale bytes) of float64 (rows, cols), from the definition."""
    rows, cols = x.shape
    wide = -(-cols // 32) * 32
    full = torch.zeros(rows, wide, dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    amax = full.reshape(rows, wide // 32, 32).abs().max(dim=2).values
    _, e = torch.frexp(amax)  # amax = f 2^e, 1/2 <= f < 1
    s = torch.where(amax > 0, (e - 1 - FORMATS[fmt][0] + 127).clamp(min=0), 0)
    inv = torch.pow(2.0, (127 - s).double()).repeat_interleave(32, dim=1)
    return _nearest(full * inv, fmt)[:, :cols], s


def _values64(q, s):
    return q * torch.pow(2.0, s.double() - 127).repeat_interleave(32, dim=1)[:, :q.shape[1]]


def _held64(codes, scales, cols, fmt):
    """float64 values of packed rows, looked up code by code."""
    pos = _positive_values(fmt)
    half = 8 if fmt == "e2m1" else 128
    pos = pos + [float("nan")] * (half - len(pos))
    table = torch.tensor(pos + [-v for v in pos], dtype=torch.float64, device=codes.device)
    i = codes.to(torch.int64)
    if fmt == "e2m1":
        i = torch.cat(((i % 16).unsqueeze(2), (i // 16).unsqueeze(2)), dim=2).flatten(1)
    return _values64(table[i], scales)[:, :cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = st["x"].double() + st["residual"].double()
        h16 = h.to(TYPES[case["type"]]).double()  # the sum of two 16-bit values is exact in 64
        mean = torch.einsum("rc,rc->r", h16, h16) / case["cols"]
        y = h16 * ((mean + EPS) ** -0.5)[:, None] * st["weight"].double()[None, :]
        if case["mx"]:
            q, s = _quantise64(y, "e4m3")
            return {"h": h, "y": {"codes": q, "scales": torch.pow(2.0, s.double() - 127)}}
        return {"h": h, "y": y}
    if op == "norm_grad":
        dy, h, w, r = (st[k].double() for k in ("dy", "h", "weight", "rstd"))
        xhat = h * r[:, None]
        g = dy * w[None, :]
        along = torch.einsum("rc,rc->r", g, xhat) / case["cols"]
        dx = (g - xhat * along[:, None]) * r[:, None]
        if case["dh"]:
            dx = dx + st["dh"].double()
        return {"dx": dx, "dweight": torch.einsum("rc,rc->c", dy, xhat)}
    if op == "quantize":
        q, s = _quantise64(st["x"].double(), case["fmt"])
        if case["fmt"] == "e4m3":
            return {"codes": q, "scales": torch.pow(2.0, s.double() - 127)}
        return {"values": _values64(q, s)}
    w = _held64(st["codes"], st["scales"], case["m"], "e2m1")
    if op == "linear":
        if case["ready"]:
            x = _held64(st["xcodes"], st["xscales"], case["m"], case["act"])
        else:
            x = _values64(*_quantise64(st["x"].double(), case["act"]))
        return {"y": torch.mm(x, w.t())}
    return {"dx": torch.mm(st["dy"].double(), w)}
