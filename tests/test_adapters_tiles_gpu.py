"""GPU: adapters whose groups fill several 16-row tiles (32 rows of a group at least, 2^22 elements of each side), at
every number of rank tiles, widths that are multiples of eight and others, against 64 bits on the device.

* whole numbers, whose sums are exact: bit for bit;
* normal data, with the tolerances of the small sizes (their derivation: test_adapters_gpu.py).

Every case prints its name before it touches the GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf

pytestmark = pytest.mark.gpu

SIZES = [  # rows, groups, n, m, rank
    (8192, 1, 520, 1032, 16), (2500, 3, 1701, 2003, 16), (700, 20, 6016, 6100, 8), (1999, 7, 2184, 4104, 24),
    (1999, 7, 2131, 2207, 32), (2048, 8, 2056, 2112, 64), (1777, 5, 2501, 2403, 48), (2048, 2, 2048, 4096, 128),
    (3001, 11, 1403, 1411, 100), (4500, 1, 1000, 935, 128),
]


def _case(rows, count, n, m, rank, name, make):
    import torch
    print(f"[case] adapters tiles {rows} rows of {count}, {n} x {m}, rank {rank}, {name}, {make.__name__}", flush=True)
    assert rows // min(rows, count) >= 32 and rows * min(n, m) >= 2 ** 22
    T = {"f16": torch.float16, "bf16": torch.bfloat16}[name]
    gen = torch.Generator(device="cuda").manual_seed(rows + n + rank)
    part = np.random.default_rng(rows).random(count + 1) + 0.2  # groups of uneven sizes, some rows of none
    part[count] *= 0.2
    sizes = (rows * part / part.sum()).astype(int)[:count]
    index = torch.full((rows,), -1, dtype=torch.int32)
    index[:sizes.sum()] = torch.repeat_interleave(torch.arange(count, dtype=torch.int32), torch.from_numpy(sizes))
    index = index.cuda()[torch.randperm(rows, generator=gen, device="cuda")].contiguous()
    v = make(torch, gen, rows, count, n, m, rank)
    v = {k: a.to(torch.float32 if k in ("t", "scale") else T) for k, a in v.items()}
    on = [torch.nonzero(index == a).flatten() for a in range(count)]
    none = torch.nonzero(index < 0).flatten()
    return T, v, {k: a.double() for k, a in v.items()}, dbf.group_rows(index, count), on, none


def whole(torch, gen, rows, count, n, m, rank):
    draw = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=gen, device="cuda").float()  # noqa: E731
    return {"x": draw(-2, 2, rows, m), "dy": draw(-2, 2, rows, n), "base": draw(-9, 9, rows, n), "dx": draw(-9, 9, rows, m),
            "A": draw(-1, 1, count, rank, m), "B": draw(-1, 1, count, n, rank), "t": draw(-500, 500, rows, rank),
            "scale": 2.0 ** draw(-1, 1, count)}


def normal(torch, gen, rows, count, n, m, rank):
    draw = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    return {"x": draw(rows, m), "dy": draw(rows, n) * 0.01, "base": draw(rows, n), "dx": draw(rows, m) * 0.01,
            "A": draw(count, rank, m) / m ** 0.5, "B": draw(count, n, rank) * 0.1, "t": draw(rows, rank),
            "scale": 0.25 + 1.75 * torch.rand(count, generator=gen, device="cuda")}


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,count,n,m,rank", SIZES)
def test_whole_numbers(gpu, rows, count, n, m, rank, name):
    import torch
    T, v, d, g, on, none = _case(rows, count, n, m, rank, name, whole)
    ad = dbf.Adapters(v["A"], v["B"], v["scale"])
    y, t = ad(v["x"], v["base"], g)
    out, dA, dB = ad.backward(v["dy"], v["x"], v["t"], g, dx=v["dx"])
    assert torch.equal(y[none], v["base"][none]) and torch.equal(out[none], v["dx"][none]) and not bool(t[none].any())
    for a, at in enumerate(on):
        A, B, s = d["A"][a], d["B"][a], d["scale"][a]
        low, u = d["x"][at] @ A.t(), s * (d["dy"][at] @ B)
        # (every sum a multiple of a half below 2^23, t and u of 16 bits at most: exact whatever the order)
        assert max(float(low.abs().max()), float(u.abs().max())) < 2 ** 15
        for got, ref in ((t[at], low), (y[at], d["base"][at] + s * (low @ B.t())), (out[at], d["dx"][at] + u @ A),
                         (dA[a], u.t() @ d["x"][at]), (dB[a], s * (d["dy"][at].t() @ d["t"][at]))):
            assert float(ref.abs().max()) < 2 ** 22
            assert torch.equal(got, ref.float().to(got.dtype))


def _within(got, ref, tol, what):
    d = (got.double() - ref).abs()
    assert bool((d <= tol).all()), f"{what}: worst {float((d / tol.clamp_min(1e-300)).max()):.3f} of the tolerance"


def _loose(size, name, sums):
    """What the 16-bit parts of values of these sizes (a group's rows x ranks) may lose."""
    if name == "bf16":
        return 2.0 ** (-25 if sums else -17) * size
    top = size.max() if sums else size.max(dim=1, keepdim=True).values
    return 2.0 ** -23 * size + 2.0 ** -38 * top


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,count,n,m,rank", SIZES)
def test_normal_data(gpu, rows, count, n, m, rank, name):
    import torch
    T, v, d, g, on, none = _case(rows, count, n, m, rank, name, normal)
    ad = dbf.Adapters(v["A"], v["B"], v["scale"])
    y, t = ad(v["x"], v["base"], g)
    out, dA, dB = ad.backward(v["dy"], v["x"], v["t"], g, dx=v["dx"])
    assert torch.equal(y[none], v["base"][none]) and torch.equal(out[none], v["dx"][none])
    half, eps = torch.finfo(T).eps / 2, 2.0 ** -24
    tiny = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]

    def rounded(got, base, w, low, te, what):
        """got = rne(base + low wᵀ) where low is off by te."""
        size = low.abs() + te
        err = (te + _loose(size, name, False) + (2 * rank / 8 + 16) * eps * size) @ w.abs().t()
        ref = base + low @ w.t()
        err = err + eps * ref.abs()
        _within(got, ref, err + half * (ref.abs() + err) + tiny, what)

    for a, at in enumerate(on):
        A, B, s, x, dy, ts = d["A"][a], d["B"][a], d["scale"][a], d["x"][at], d["dy"][at], d["t"][at]
        low, te = x @ A.t(), (m / 8 + 16) * eps * (x.abs() @ A.abs().t())
        _within(t[at], low, te, "t")
        rounded(y[at], d["base"][at], s * B, low, te, "y")
        u, ue = s * (dy @ B), (n / 8 + 17) * eps * s * (dy.abs() @ B.abs())
        rounded(out[at], d["dx"][at], A.t(), u, ue, "dx")
        sums = (3 * rows / 8 + 20) * eps
        size = u.abs() + ue
        _within(dA[a], u.t() @ x, (ue + _loose(size, name, True) + sums * size).t() @ x.abs() + 2.0 ** -149, "dA")
        _within(dB[a], s * (dy.t() @ ts), s * (dy.abs().t() @ (_loose(ts.abs(), name, True) + sums * ts.abs())) + 2.0 ** -149, "dB")
    again = v["base"].clone()
    assert torch.equal(ad(v["x"], again, g, out=again).y, y)
    again = v["dx"].clone()
    second = ad.backward(v["dy"], v["x"], v["t"], g, dx=again, out=again)
    assert all(torch.equal(p, q) for p, q in zip(second, (out, dA, dB)))
