"""Cases of the operators on rows that belong to groups, for measurement: the sorting of rows by group, the
products of 4-bit experts and their input gradients, and the low-rank adapters beside a layer with their gradients.

run() computes a case in its plain form (elementary torch operations in 32
bits, one rounding at the end) or, where `own` is true, by the calls that a
program makes of this package.  exact() gives the same outputs from the
operators' definitions in 64 bits.

An index assigns each of its rows (slots) to one of `count` groups; -1 is no
group.  Slots in the order of their groups, each group's in rising order and
those of no group last, are the grouped order.  The block format of the
experts' weights and inputs: 32 consecutive columns of a row share one
power-of-two scale (a byte s, 2^(s-127)) and hold e4m3 or e2m1 codes; rows are
padded with zero bytes to a multiple of 128 columns, e2m1 holds two codes in a
byte, the even column in the low half.
"""

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # sixteen decoded tokens, eight of 64 experts each
        {"name": "group_decode", "op": "group", "tokens": 16, "top": 8, "count": 64, "none": 0.0},
        # a prompt's tokens, the batch padded at its end
        {"name": "group_prompt", "op": "group", "tokens": 2048, "top": 8, "count": 64, "none": 0.1},
        # one token through the up projections of two of eight experts
        {"name": "experts_one_token", "op": "experts", "tokens": 1, "top": 2, "count": 8, "n": 14336, "m": 4096,
         "type": "f16", "act": "e4m3", "ready": False, "side": "up", "none": 0.0},
        # sixteen sequences decoded together, down projections of many small experts
        {"name": "experts_decode_batch", "op": "experts", "tokens": 16, "top": 8, "count": 64, "n": 4096, "m": 1024,
         "type": "bf16", "act": "e4m3", "ready": False, "side": "down", "none": 0.0},
        # a prompt through the up projections, rows quantised in the call
        {"name": "experts_prompt", "op": "experts", "tokens": 2048, "top": 2, "count": 8, "n": 14336, "m": 4096,
         "type": "bf16", "act": "e4m3", "ready": False, "side": "up", "none": 0.0},
        # odd sizes, 4-bit rows, a padded batch
        {"name": "experts_ragged", "op": "experts", "tokens": 333, "top": 4, "count": 13, "n": 1000, "m": 1300,
         "type": "f16", "act": "e2m1", "ready": True, "side": "up", "none": 0.1},
        # fine-tuning through frozen experts: the input's gradient of the up projections
        {"name": "experts_grad_prompt", "op": "experts_grad", "tokens": 2048, "top": 2, "count": 8, "n": 14336,
         "m": 4096, "type": "bf16", "none": 0.0},
        # the same at odd sizes
        {"name": "experts_grad_ragged", "op": "experts_grad", "tokens": 77, "top": 3, "count": 13, "n": 1000,
         "m": 1300, "type": "f16", "none": 0.1},
        # sixteen requests decoded together, each with its own adapter or none, beside a square projection
        {"name": "adapters_decode", "op": "adapters", "rows": 16, "count": 32, "n": 4096, "m": 4096, "rank": 16,
         "type": "f16", "runs": False, "none": 0.1},
        # prompts of several requests in one batch, beside an up projection
        {"name": "adapters_prompt", "op": "adapters", "rows": 2048, "count": 8, "n": 14336, "m": 4096, "rank": 64,
         "type": "bf16", "runs": True, "none": 0.0},
        # fine-tuning one adapter over a batch of sequences
        {"name": "adapters_grad_batch", "op": "adapters_grad", "rows": 8192, "count": 1, "n": 4096, "m": 4096,
         "rank": 16, "type": "bf16", "runs": True, "none": 0.0},
        # several adapters tuned together, at odd sizes
        {"name": "adapters_grad_ragged", "op": "adapters_grad", "rows": 300, "count": 5, "n": 1000, "m": 1300,
         "rank": 24, "type": "f16", "runs": True, "none": 0.1},
    ]


def _spread(rng, low, high):
    """A whole number of [low, high], even over its logarithm; half of them a multiple of 64 where that fits."""
    v = int(round(low * (high / low) ** rng.random()))
    if rng.random() < 0.5 and v >= 64:
        v = v // 64 * 64
    return max(low, min(high, v))


def draw(rng):
    op = rng.choice(["group", "experts", "experts", "experts", "experts_grad", "adapters", "adapters",
                     "adapters_grad"])
    none = rng.choice([0.0, 0.1])
    if op == "group":
        count = _spread(rng, 2, 256)
        return {"op": op, "tokens": _spread(rng, 1, 8192), "top": min(count, rng.randint(1, 8)), "count": count,
                "none": none}
    n, m = _spread(rng, 64, 14336), _spread(rng, 64, 14336)
    t = rng.choice(["f16", "bf16"])
    if op in ("experts", "experts_grad"):
        count = _spread(rng, 2, 128)
        while count * n * m > 8 * 14336 * 4096:
            if n > m:
                n = max(64, n // 2)
            else:
                m = max(64, m // 2)
        c = {"op": op, "tokens": _spread(rng, 1, 2048), "top": min(count, rng.randint(1, 8)), "count": count, "n": n,
             "m": m, "type": t, "none": none}
        while c["tokens"] * c["top"] * n * m > 2048 * 2 * 14336 * 4096:
            c["tokens"] = max(1, c["tokens"] // 2)
        if op == "experts":
            c["act"] = rng.choice(["e4m3", "e2m1"])
            c["ready"] = rng.random() < 0.4
            c["side"] = rng.choice(["up", "down"])
        return c
    c = {"op": op, "rows": _spread(rng, 1, 8192), "count": _spread(rng, 1, 64), "n": n, "m": m,
         "rank": rng.choice([4, 8, 16, 24, 32, 64, 128]), "type": t, "runs": rng.random() < 0.6, "none": none}
    while c["rows"] * (n + m) > 2048 * (14336 + 4096):
        c["rows"] = max(1, c["rows"] // 2)
    return c


def work(case):
    op, count = case["op"], case["count"]
    if op == "group":
        s = case["tokens"] * case["top"]
        return {"bytes": 8 * s + 4 * (count + 1), "flops": s}
    n, m = case["n"], case["m"]
    if op in ("experts", "experts_grad"):
        s = case["tokens"] * case["top"]
        used = min(count, s)
        weight = used * (n * m // 2 + n * m // 32)
        if op == "experts_grad":
            return {"bytes": weight + 2 * s * (n + m) + 4 * s, "flops": 2 * s * n * m}
        size = 2 if not case["ready"] else 33 / 32 if case["act"] == "e4m3" else 17 / 32
        rows = case["tokens"] if case["side"] == "up" else s
        return {"bytes": weight + rows * m * size + 2 * s * n + 4 * s, "flops": 2 * s * n * m}
    s, r = case["rows"], case["rank"]
    factors = min(count, s) * r * (n + m)
    if op == "adapters":
        return {"bytes": 2 * factors + 2 * s * (m + 2 * n) + 4 * s * r + 4 * s, "flops": 2 * s * r * (n + m)}
    return {"bytes": 2 * factors + 4 * count * r * (n + m) + 2 * s * (n + 3 * m) + 4 * s * r + 4 * s,
            "flops": 4 * s * r * (n + m)}


# ------------------------------------------------------- the block format, plain

# format: largest value's exponent, mantissa bits, smallest normal exponent, largest value
FORMATS = {"e4m3": (8, 3, -6, 448.0), "e2m1": (2, 1, 0, 6.0)}


def _exponent(x):
    """floor(log2 |x|) of float32 values (normal ones; -127 and below for the rest)."""
    return ((x.view(torch.int32) >> 23) & 255) - 127


def _quantise(x, fmt):
    """(codes as the values they stand for, before the scale; scale bytes) of finite float32 (rows, cols)."""
    emax, mant, emin, top = FORMATS[fmt]
    rows, cols = x.shape
    b = torch.nn.functional.pad(x, (0, -cols % 32)).reshape(rows, (cols + 31) // 32, 32)
    s = (_exponent(b.abs().amax(dim=2)) - emax + 127).clamp(0, 254)
    v = torch.ldexp(b, 127 - s.unsqueeze(2))
    step = torch.ldexp(torch.ones_like(v), _exponent(v).clamp(min=emin) - mant)
    q = (torch.round(v / step) * step).clamp(-top, top)
    return q.reshape(rows, -1)[:, :cols], s


def _values(q, s):
    scale = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.to(torch.int32) - 127)
    return q * scale.repeat_interleave(32, dim=1)[:, :q.shape[1]]


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


def _routes(gen, case):
    """int32 index of tokens * top slots: each token's experts of largest score, some experts more popular than
    others; the last tokens of a padded batch have none."""
    dev, tokens, count = gen.device, case["tokens"], case["count"]
    score = torch.randn(tokens, count, generator=gen, device=dev) + 0.7 * torch.randn(count, generator=gen, device=dev)
    ids = score.topk(case["top"], dim=1).indices.to(torch.int32)
    ids[tokens - int(case["none"] * tokens):] = -1
    return ids.flatten()


def _requests(gen, case):
    """int32 index of rows: the adapter of each row's request, -1 for those without one."""
    dev, rows, count = gen.device, case["rows"], case["count"]
    which = torch.randint(0, count, (rows,), generator=gen, device=dev)
    which = torch.where(torch.rand(rows, generator=gen, device=dev) < case["none"], -1, which)
    if case["runs"]:  # sequences of many rows, one adapter each
        starts = torch.rand(rows, generator=gen, device=dev) < 4 * max(count, 2) / max(rows, 1)
        which = which[starts.cumsum(0).clamp(max=rows - 1)]
    return which.to(torch.int32)


def _host_groups(index, count):
    """(grouped order of the slots, list of the groups' first places and the end of the last)."""
    key = torch.where(index < 0, count, index)
    order = torch.sort(key, stable=True).indices
    ends = torch.searchsorted(key[order].contiguous(), torch.arange(count + 1, device=index.device, dtype=key.dtype))
    return order, ends.tolist()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dev, op, count = gen.device, case["op"], case["count"]
    st = {"case": case}
    if op == "group":
        st["index"] = _routes(gen, case)
        return st
    n, m, t = case["n"], case["m"], TYPES[case["type"]]
    if op in ("experts", "experts_grad"):
        index = _routes(gen, case)
        slots = index.numel()
        parts = []
        for _ in range(count):
            parts.append(_pack(*_quantise(0.02 * torch.randn(n, m, generator=gen, device=dev), "e2m1"), "e2m1"))
        st["codes"] = torch.cat([p[0] for p in parts])
        st["scales"] = torch.cat([p[1] for p in parts])
        del parts
        if op == "experts_grad":
            # in grouped order, as the activation's gradient leaves it
            st["dy"] = (0.01 * torch.randn(slots, n, generator=gen, device=dev)).to(t)
        else:
            # up: a row per token; down: a row per slot, in grouped order
            x = _activations(gen, case["tokens"] if case["side"] == "up" else slots, m, t)
            if case["ready"]:
                st["xcodes"], st["xscales"] = _pack(*_quantise(x.float(), case["act"]), case["act"])
            else:
                st["x"] = x
        # the largest number of slots that the program routes at once
        st["slots"] = slots
    else:
        index = _requests(gen, case)
        s, r = case["rows"], case["rank"]
        st["x"] = _activations(gen, s, m, t)
        st["A"] = (torch.randn(count, r, m, generator=gen, device=dev) / m ** 0.5).to(t)
        st["B"] = (0.05 * torch.randn(count, n, r, generator=gen, device=dev)).to(t)
        st["scale"] = 0.5 + 1.5 * torch.rand(count, generator=gen, device=dev)
        if op == "adapters":
            st["base"] = torch.randn(s, n, generator=gen, device=dev).to(t)
        else:
            st["dy"] = (0.01 * torch.randn(s, n, generator=gen, device=dev)).to(t)
            st["dx"] = (0.01 * torch.randn(s, m, generator=gen, device=dev)).to(t)
            # kept from the forward pass
            tt = torch.zeros(s, r, dtype=torch.float64, device=dev)
            for e in range(count):
                at = (index == e).nonzero().flatten()
                tt[at] = st["x"][at].double() @ st["A"][e].double().t()
            st["t"] = tt.float()
    # the groups are sorted once for all layers that the rows pass
    st["order"], st["ends"] = _host_groups(index, count)
    if own:
        import dbf_linear_fwd_amd as dbf
        st["groups"] = dbf.group_rows(index, count)
        if op in ("experts", "experts_grad"):
            st["layer"] = dbf.Experts(dbf.MxTensor(st["codes"], st["scales"], m, "e2m1"), count,
                                      max_rows=st["slots"], act=case.get("act", "e4m3"))
        else:
            st["layer"] = dbf.Adapters(st["A"], st["B"], st["scale"])
    return st


# ------------------------------------------------------------------ one pass

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import dbf_linear_fwd_amd as dbf
    case = st["case"]
    op = case["op"]
    if op == "group":
        g = dbf.group_rows(st["index"], case["count"])
        return {"order": g.order, "offsets": g.offsets}
    if op == "experts":
        x = dbf.MxTensor(st["xcodes"], st["xscales"], case["m"], case["act"]) if case["ready"] else st["x"]
        up = case["side"] == "up"
        # up: tokens in, grouped order out; down: grouped order in, slots in the index's order out
        return {"y": st["layer"].forward(x, st["groups"], gather=case["top"] if up else 0, scatter=not up,
                                         out_dtype=TYPES[case["type"]])}
    if op == "experts_grad":
        # back to the index's order, where a token's slots are added up
        return {"dx": st["layer"].backward_data(st["dy"], st["groups"], scatter=True)}
    if op == "adapters":
        y, t = st["layer"].forward(st["x"], st["base"], st["groups"])
        return {"y": y, "t": t}
    dx, dA, dB = st["layer"].backward(st["dy"], st["x"], st["t"], st["groups"], dx=st["dx"])
    return {"dx": dx, "dA": dA, "dB": dB}


def _run_plain(st):
    case = st["case"]
    op, count = case["op"], case["count"]
    if op == "group":
        index = st["index"]
        key = torch.where(index < 0, count, index)
        order = torch.sort(key, stable=True).indices
        groups = torch.arange(count, device=index.device, dtype=key.dtype)
        sizes = (key.unsqueeze(1) == groups).sum(dim=0)
        offsets = torch.nn.functional.pad(sizes.cumsum(0), (1, 0))
        return {"order": order.to(torch.int32), "offsets": offsets.to(torch.int32)}
    n, m, t = case["n"], case["m"], TYPES[case["type"]]
    order, ends = st["order"], st["ends"]
    if op in ("experts", "experts_grad"):
        def weight(e):
            rows = slice(e * n, (e + 1) * n)
            return _unpack(st["codes"][rows], st["scales"][rows], m, "e2m1")
        if op == "experts_grad":
            dx = torch.zeros(order.numel(), m, dtype=t, device=order.device)
            for e in range(count):
                lo, hi = ends[e], ends[e + 1]
                if hi > lo:
                    dx[order[lo:hi]] = (st["dy"][lo:hi].float() @ weight(e)).to(t)
            return {"dx": dx}
        if case["ready"]:
            x = _unpack(st["xcodes"], st["xscales"], m, case["act"])
        else:
            x = _values(*_quantise(st["x"].float(), case["act"]))
        y = torch.zeros(order.numel(), n, dtype=t, device=order.device)
        for e in range(count):
            lo, hi = ends[e], ends[e + 1]
            if hi == lo:
                continue
            if case["side"] == "up":
                y[lo:hi] = (x[order[lo:hi] // case["top"]] @ weight(e).t()).to(t)
            else:
                y[order[lo:hi]] = (x[lo:hi] @ weight(e).t()).to(t)
        return {"y": y}
    if op == "adapters":
        y = st["base"].clone()
        low = torch.zeros(case["rows"], case["rank"], dtype=torch.float32, device=y.device)
        for e in range(count):
            lo, hi = ends[e], ends[e + 1]
            if hi == lo:
                continue
            at = order[lo:hi]
            te = st["x"][at].float() @ st["A"][e].float().t()
            low[at] = te
            y[at] = (st["base"][at].float() + st["scale"][e] * (te @ st["B"][e].float().t())).to(t)
        return {"y": y, "t": low}
    dx = st["dx"].clone()
    dA = torch.zeros(st["A"].shape, dtype=torch.float32, device=dx.device)
    dB = torch.zeros(st["B"].shape, dtype=torch.float32, device=dx.device)
    for e in range(count):
        lo, hi = ends[e], ends[e + 1]
        if hi == lo:
            continue
        at = order[lo:hi]
        g, x = st["dy"][at].float(), st["x"][at].float()
        u = st["scale"][e] * (g @ st["B"][e].float())
        dx[at] = (st["dx"][at].float() + u @ st["A"][e].float()).to(t)
        dA[e] = u.t() @ x
        dB[e] = st["scale"][e] * (g.t() @ st["t"][at])
    return {"dx": dx, "dA": dA, "dB": dB}


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


def _blocks64(x, fmt):
    """Values of float64 (rows, cols) after the format's rounding, from the definition."""
    rows, cols = x.shape
    nb = (cols + 31) // 32
    full = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    full[:, :cols] = x
    b = full.view(rows, nb, 32)
    _, e = torch.frexp(b.abs().max(dim=2, keepdim=True).values)  # amax = f 2^e, 1/2 <= f < 1
    s = (e - 1 - FORMATS[fmt][0]).clamp(min=-127).double()
    return (_nearest(b * torch.pow(2.0, -s), fmt) * torch.pow(2.0, s)).view(rows, nb * 32)[:, :cols]


def _held64(codes, scales, cols, fmt):
    """float64 values of packed rows, looked up code by code."""
    pos = _positive_values(fmt)
    half = 8 if fmt == "e2m1" else 128
    pos = pos + [float("nan")] * (half - len(pos))
    table = torch.tensor(pos + [-v for v in pos], dtype=torch.float64, device=codes.device)
    i = codes.to(torch.int64)
    if fmt == "e2m1":
        i = torch.cat(((i % 16).unsqueeze(2), (i // 16).unsqueeze(2)), dim=2).flatten(1)
    q = table[i]
    return (q.view(q.shape[0], -1, 32) * torch.pow(2.0, scales.double() - 127).unsqueeze(2)).view(q.shape)[:, :cols]



def exact(case, seed):
    op, count = case["op"], case["count"]
    st = prepare(case, seed)
    if op == "group":
        index = st["index"].tolist()
        lists = [[] for _ in range(count + 1)]
        for j, v in enumerate(index):
            lists[v if v >= 0 else count].append(j)
        offsets = [0]
        for part in lists[:count]:
            offsets.append(offsets[-1] + len(part))
        dev = st["index"].device
        return {"order": torch.tensor([j for part in lists for j in part], dtype=torch.int32, device=dev),
                "offsets": torch.tensor(offsets, dtype=torch.int32, device=dev)}
    n, m = case["n"], case["m"]
    # the group of every place of the grouped order, and the place's slot
    order, ends = st["order"], st["ends"]
    dev = order.device
    where = torch.arange(order.numel(), device=dev)
    if op in ("experts", "experts_grad"):
        grad = op == "experts_grad"
        up = not grad and case["side"] == "up"
        if grad:
            x = st["dy"].double()
        elif case["ready"]:
            x = _held64(st["xcodes"], st["xscales"], m, case["act"])
        else:
            x = _blocks64(st["x"].double(), case["act"])
        out = torch.zeros(order.numel(), m if grad else n, dtype=torch.float64, device=dev)
        for e in range(count):
            mine = (where >= ends[e]) & (where < ends[e + 1])
            if ends[e + 1] == ends[e]:
                continue
            w = _held64(st["codes"][e * n:(e + 1) * n], st["scales"][e * n:(e + 1) * n], m, "e2m1")
            rows = torch.div(order[mine], case["top"], rounding_mode="floor") if up else where[mine]
            out[where[mine] if up else order[mine]] = torch.mm(x[rows], w if grad else w.t())
        return {"dx" if grad else "y": out}
    r = case["rank"]
    scale = st["scale"].double()
    x = st["x"].double()
    if op == "adapters":
        y, low = st["base"].double(), torch.zeros(case["rows"], r, dtype=torch.float64, device=dev)
        for e in range(count):
            at = order[ends[e]:ends[e + 1]]
            if at.numel():
                low[at] = torch.mm(x[at], st["A"][e].double().t())
                y[at] += torch.mm(low[at], (scale[e] * st["B"][e].double()).t())
        return {"y": y, "t": low}
    dx = st["dx"].double()
    dA = torch.zeros(count, r, m, dtype=torch.float64, device=dev)
    dB = torch.zeros(count, n, r, dtype=torch.float64, device=dev)
    for e in range(count):
        at = order[ends[e]:ends[e + 1]]
        if at.numel():
            g = scale[e] * st["dy"][at].double()
            u = torch.mm(g, st["B"][e].double())
            dx[at] += torch.mm(u, st["A"][e].double())
            dA[e] = torch.mm(u.t(), x[at])
            dB[e] = torch.mm(g.t(), st["t"][at].double())
    return {"dx": dx, "dA": dA, "dB": dB}
