"""GPU: infinities in every operand of the adapters, forward and backward: results are infinite or NaN where the
formula's are, and only there, whatever 16-bit parts t and u have.

A product of matrices with infinities: a sum is NaN where a term is (0 * inf,
or a NaN), or where infinities of both signs meet, and infinite where one
kind of them does; the others are finite.  The terms of each kind are counted
by products of indicator matrices in 64 bits.

Every case prints its name before it touches the GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf

def product(a, b):
    """a @ b in 64 bits, infinities and NaN as IEEE's sums of products have them."""
    clean = lambda v: np.where(np.isfinite(v), v, 0.0)  # noqa: E731
    up, down, zero, nan = [], [], [], []
    for v in (a, b):
        up.append((v > 0).astype(float))
        down.append((v < 0).astype(float))
        zero.append((v == 0).astype(float))
        nan.append(np.isnan(v).astype(float))
    ia, ib = np.isinf(a), np.isinf(b)
    any_a, any_b = np.ones_like(a), np.ones_like(b)
    plus = (up[0] * ia) @ up[1] + (down[0] * ia) @ down[1] + up[0] @ (up[1] * ib) + down[0] @ (down[1] * ib)
    minus = (up[0] * ia) @ down[1] + (down[0] * ia) @ up[1] + up[0] @ (down[1] * ib) + down[0] @ (up[1] * ib)
    bad = nan[0] @ any_b + any_a @ nan[1] + (ia * 1.0) @ zero[1] + zero[0] @ (ib * 1.0)
    out = clean(a) @ clean(b)
    out = np.where(plus > 0, np.inf, out)
    out = np.where(minus > 0, -np.inf, out)
    return np.where((bad > 0) | ((plus > 0) & (minus > 0)), np.nan, out)


def test_product_by_hand():
    inf, nan = np.inf, np.nan
    a = np.array([[inf, 1.0], [-inf, 2.0], [0.0, 3.0], [1.0, 1.0]])
    b = np.array([[2.0, 0.0, inf], [1.0, 1.0, -inf]])
    got, want = product(a, b), np.array([[inf, nan, nan], [-inf, nan, -inf], [3.0, 3.0, nan], [3.0, 1.0, nan]])
    assert np.array_equal(got, want, equal_nan=True)


def check(got, ref, mag, K, half, what):
    got = got.double().cpu().numpy()
    for kind in (np.isnan, np.isposinf, np.isneginf):
        d = kind(got) != kind(ref)
        assert not d.any(), f"{what}: {kind.__name__} differs at {np.argwhere(d)[:3].tolist()} of {d.sum()}"
    ok = np.isfinite(ref)
    # half a step, t's or u's 16-bit parts, and at most K / 8 + 40 roundings of the sums
    tol = (half + 2.0 ** -24) * np.abs(ref[ok]) + (2.0 ** -16 + (K / 8 + 40) * 2.0 ** -24) * mag[ok] + 1e-30
    assert np.all(np.abs(got[ok] - ref[ok]) <= tol), what


def values(rng, shape):
    """Whole multiples of 1/4 up to 2, some zeros: one 16-bit part holds them."""
    v = rng.integers(1, 9, size=shape) / 4.0 * rng.choice([-1.0, 1.0], size=shape)
    return np.where(rng.random(shape) < 0.02, 0.0, v)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [3, 16, 20, 40, 100])
@pytest.mark.parametrize("rows,n,m", [(7, 72, 140), (70, 133, 75), (600, 7200, 7104)])
@pytest.mark.parametrize("where", ["x", "dy", "A", "B", "t", "none"])
def test_infinite_operands(gpu, where, rows, n, m, rank, name):
    import torch
    print(f"[case] infinities in {where}: {rows} rows, n {n}, m {m}, rank {rank}, {name}", flush=True)
    T = {"f16": torch.float16, "bf16": torch.bfloat16}[name]
    half = torch.finfo(T).eps / 2
    rng = np.random.default_rng(rank + n + len(where))
    v = {"x": values(rng, (rows, m)), "dy": values(rng, (rows, n)), "A": values(rng, (rank, m)),
         "B": values(rng, (n, rank)), "t": values(rng, (rows, rank))}
    if where != "none":
        a = v[where]
        for k, (i, j) in enumerate(((1, 1), (2, 0), (a.shape[0] - 1, a.shape[1] - 1))):
            a[i, j] = np.inf if k != 1 else -np.inf
    dev = lambda k: torch.from_numpy(v[k]).to(T).cuda()  # noqa: E731
    ad = dbf.Adapters(dev("A")[None], dev("B")[None])
    g = dbf.group_rows(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1)
    mag = {k: np.where(np.isfinite(a), np.abs(a), 0.0) for k, a in v.items()}
    if where in ("x", "A", "B", "none"):
        y, t = ad(dev("x"), torch.zeros(rows, n, dtype=T, device="cuda"), g)
        low = product(v["x"], v["A"].T)
        check(t, low, mag["x"] @ mag["A"].T, m, 0.0, "t")
        check(y, product(low, v["B"].T), (mag["x"] @ mag["A"].T) @ mag["B"].T, m, half, "y")
    dx, dA, dB = ad.backward(dev("dy"), dev("x"), torch.from_numpy(v["t"]).float().cuda(), g)
    u, um = product(v["dy"], v["B"]), mag["dy"] @ mag["B"]
    check(dx, product(u, v["A"]), um @ mag["A"], n, half, "dx")
    check(dA[0], product(u.T, v["x"]), um.T @ mag["x"], n + 3 * rows, 0.0, "dA")
    check(dB[0], product(v["dy"].T, v["t"]), mag["dy"].T @ mag["t"], 3 * rows, 0.0, "dB")
