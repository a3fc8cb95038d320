"""GPU: low-rank adapters and their gradients, against the fp64 oracle.

Tolerances.  A product of 16-bit values is exact in fp32.  The matrix core adds
the 32 products of an instruction in partial sums of eight at least, each
rounded once, so a sum over K has at most K / 8 + 16 roundings (joins of waves
and parts included) of 2^-24 of Σ|a b|.  t and u enter the second products in
16-bit parts: bf16 two parts, 2^-17 of each value (three, 2^-25, in dA and dB);
f16 two, 2^-23 of each value or 2^-38 of the largest that shares its power of two
(the row's, in dA and dB the group's).  The result is rounded once: half a step.

Every case prints its name before it touches the GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import rows_oracle as O

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)


def _torch():
    import torch
    return torch


def T(name):
    torch = _torch()
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def tiny(name):
    return {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]


def to_dev(x, name):
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).to(T(name))
    return t.cuda(), t.double().numpy()


def group(index, count):
    torch = _torch()
    return dbf.group_rows(torch.from_numpy(np.asarray(index)).to(torch.int32).cuda(), count)


def spread(rng, rows, count, none=0.1):
    v = np.where(rng.random(rows) < 0.4, rng.integers(0, count), rng.integers(0, count, rows))
    return np.where(rng.random(rows) < none, -1, v)


def within(got, ref, tol, what):
    d = np.abs(got - ref)
    assert np.all(d <= tol), f"{what}: worst {float((d / np.maximum(tol, 1e-300)).max()):.3f} of the tolerance"


def parts_error(v, index, name, sums):
    """What the 16-bit parts of v (rows x rank) may lose; sums: in the products over a group's rows."""
    if name == "bf16":
        return 2.0 ** (-25 if sums else -17) * np.abs(v)
    top = np.abs(v).max(axis=1, keepdims=True)
    if sums:
        for a in set(index):
            at = [r for r, i in enumerate(index) if i == a]
            top[at] = top[at].max()
    return 2.0 ** -23 * np.abs(v) + 2.0 ** -38 * top


SIZES = [  # rows, count, n, m, rank
    (1, 1, 8, 8, 1), (1, 3, 64, 128, 16), (2, 2, 33, 40, 5), (16, 32, 256, 512, 16), (17, 4, 100, 257, 8),
    (70, 3, 300, 96, 24), (130, 1, 520, 1000, 32), (200, 5, 72, 264, 64), (300, 2, 1000, 1300, 100),
    (64, 2, 264, 2056, 128), (500, 1024, 16, 24, 4), (700, 2, 130, 66, 48), (9, 70, 40, 4096, 12),
    (3, 1, 4096, 24, 17), (1500, 3, 256, 128, 16),
]


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,count,n,m,rank", SIZES)
def test_forward(gpu, rows, count, n, m, rank, name):
    _say(f"adapters {rows} rows {count} x ({n} x {m}) rank {rank} {name}")
    rng = np.random.default_rng(rows + n + rank)
    index = spread(rng, rows, count)
    x, xv = to_dev(rng.standard_normal((rows, m)), name)
    base, bv = to_dev(rng.standard_normal((rows, n)), name)
    A, Av = to_dev(rng.standard_normal((count, rank, m)) / m ** 0.5, name)
    B, Bv = to_dev(rng.standard_normal((count, n, rank)) * 0.1, name)
    scale = rng.uniform(0.25, 2.0, count).astype(np.float32)
    ad = dbf.Adapters(A, B, _torch().from_numpy(scale).cuda())
    g = group(index, count)
    y, t = ad(x, base, g)
    yr, tr = O.adapters(xv, bv, Av, Bv, scale.astype(np.float64), index)
    _, tm = O.adapters(np.abs(xv), np.abs(bv), np.abs(Av), np.abs(Bv), scale.astype(np.float64), index)
    te = (m / 8 + 16) * 2.0 ** -24 * tm
    within(t.double().cpu().numpy(), tr, te, "t")
    # the same through B: what t is off by, its parts, the sums, and scale * t rounded
    loose = te + parts_error(np.abs(tr) + te, index, name, False) + (2 * rank / 8 + 16) * 2.0 ** -24 * (np.abs(tr) + te)
    ye = np.zeros_like(yr)
    for r, a in enumerate(index):
        if a >= 0:
            ye[r] = scale[a] * (np.abs(Bv[a]) @ loose[r])
    ye += 2.0 ** -24 * np.abs(yr)
    half = _torch().finfo(T(name)).eps / 2
    yg = y.double().cpu().numpy()
    within(yg, yr, ye + half * (np.abs(yr) + ye) + tiny(name), "y")
    none = [r for r in range(rows) if index[r] < 0]
    assert np.array_equal(yg[none], bv[none]) and not t.cpu().numpy()[none].any()
    # in place, and again: the same bits
    again = base.clone()
    ad(x, again, g, out=again)
    assert _torch().equal(again, y)


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,count,n,m,rank", SIZES)
def test_backward(gpu, rows, count, n, m, rank, name):
    _say(f"adapters backward {rows} rows {count} x ({n} x {m}) rank {rank} {name}")
    torch = _torch()
    rng = np.random.default_rng(3 * rows + n + rank)
    index = spread(rng, rows, count)
    x, xv = to_dev(rng.standard_normal((rows, m)), name)
    dy, dyv = to_dev(rng.standard_normal((rows, n)) * 0.01, name)
    dx, dxv = to_dev(rng.standard_normal((rows, m)) * 0.01, name)
    A, Av = to_dev(rng.standard_normal((count, rank, m)) / m ** 0.5, name)
    B, Bv = to_dev(rng.standard_normal((count, n, rank)) * 0.1, name)
    scale = rng.uniform(0.25, 2.0, count).astype(np.float32)
    tv = rng.standard_normal((rows, rank)).astype(np.float32)
    t = torch.from_numpy(tv).cuda()
    tv = tv.astype(np.float64)
    ad = dbf.Adapters(A, B, torch.from_numpy(scale).cuda())
    g = group(index, count)
    out, dA, dB = ad.backward(dy, x, t, g, dx=dx)
    sv = scale.astype(np.float64)
    dxr, ur, dAr, dBr = O.adapters_backward(dyv, xv, tv, dxv, Av, Bv, sv, index)
    _, um, _, _ = O.adapters_backward(np.abs(dyv), np.abs(xv), np.abs(tv), dxv, np.abs(Av), np.abs(Bv), sv, index)
    ue = (n / 8 + 17) * 2.0 ** -24 * um
    half = torch.finfo(T(name)).eps / 2
    size = np.abs(ur) + ue
    loose = ue + parts_error(size, index, name, False) + (2 * rank / 8 + 16) * 2.0 ** -24 * size
    xe = np.zeros_like(dxr)
    for r, a in enumerate(index):
        if a >= 0:
            xe[r] = np.abs(Av[a]).T @ loose[r]
    xe += 2.0 ** -24 * np.abs(dxr)
    within(out.double().cpu().numpy(), dxr, xe + half * (np.abs(dxr) + xe) + tiny(name), "dx")
    sums = (3 * rows / 8 + 20) * 2.0 ** -24
    la = ue + parts_error(size, index, name, True) + sums * size
    lb = parts_error(tv, index, name, True) + sums * np.abs(tv)
    Ae, Be = np.zeros_like(dAr), np.zeros_like(dBr)
    for r, a in enumerate(index):
        if a >= 0:
            Ae[a] += np.outer(la[r], np.abs(xv[r]))
            Be[a] += sv[a] * np.outer(np.abs(dyv[r]), lb[r])
    within(dA.double().cpu().numpy(), dAr, Ae + 2.0 ** -149, "dA")
    within(dB.double().cpu().numpy(), dBr, Be + 2.0 ** -149, "dB")
    none = [r for r in range(rows) if index[r] < 0]
    assert np.array_equal(out.double().cpu().numpy()[none], dxv[none])
    again = dx.clone()
    second = ad.backward(dy, x, t, g, dx=again, out=again)
    assert torch.equal(second[0], out) and torch.equal(second[1], dA) and torch.equal(second[2], dB)
    # without the layer's gradient: zeros in its place
    alone, _, _ = ad.backward(dy, x, t, g)
    ref = dxr - dxv
    ae = xe + 2.0 ** -24 * np.abs(ref)
    within(alone.double().cpu().numpy(), ref, ae + half * (np.abs(ref) + ae) + tiny(name), "dx alone")


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_gradients_are_differences(gpu, name):
    """The loss Σ dy y along a direction in A, B and x, by central differences of the oracle's forward (exact in fp64
    up to the difference's own error), against the gradients."""
    _say(f"adapters differences {name}")
    torch = _torch()
    rng = np.random.default_rng(21)
    rows, count, n, m, rank = 24, 3, 40, 56, 8
    index = spread(rng, rows, count)
    x, xv = to_dev(rng.standard_normal((rows, m)), name)
    dy, dyv = to_dev(rng.standard_normal((rows, n)), name)
    A, Av = to_dev(rng.standard_normal((count, rank, m)) / 8, name)
    B, Bv = to_dev(rng.standard_normal((count, n, rank)) / 8, name)
    ad = dbf.Adapters(A, B)
    one = np.ones(count)
    base = np.zeros((rows, n))
    g = group(index, count)
    _, t = ad(x, torch.zeros(rows, n, dtype=T(name), device="cuda"), g)
    dx, dA, dB = (v.double().cpu().numpy() for v in ad.backward(dy, x, t, g))
    loss = lambda x, A, B: (O.adapters(x, base, A, B, one, index)[0] * dyv).sum()  # noqa: E731
    h = 2.0 ** -20
    for k, grad in ((0, dx), (1, dA), (2, dB)):
        v = [xv, Av, Bv]
        d = rng.standard_normal(v[k].shape)
        up, down = list(v), list(v)
        up[k], down[k] = v[k] + h * d, v[k] - h * d
        want = (loss(*up) - loss(*down)) / (2 * h)
        # dx is rounded to 16 bits; each loss is linear in each of the three, and its fp64 error below 1e-15 of its terms
        terms = np.abs(grad * d).sum()
        tol = terms * (torch.finfo(T(name)).eps if k == 0 else 2.0 ** -18) + 1e-12 * abs(loss(*v)) / h + 1e-9
        assert abs((grad * d).sum() - want) <= tol


def test_no_rows_and_empty_groups(gpu):
    torch = _torch()
    A = torch.randn(3, 4, 16, device="cuda").half()
    B = torch.randn(3, 8, 4, device="cuda").half()
    ad = dbf.Adapters(A, B)
    g = dbf.group_rows(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    x, b = A.new_empty(0, 16), A.new_empty(0, 8)
    y, t = ad(x, b, g)
    assert y.shape == (0, 8) and t.shape == (0, 4)
    dx, dA, dB = ad.backward(b, x, t, g)
    assert dx.shape == (0, 16) and not bool(dA.any()) and not bool(dB.any())
    # no row of any adapter: the layer's results and gradients as they are, -0 and NaN too
    g = group(np.full(20, -1), 3)
    x = torch.full((20, 16), float("nan"), device="cuda").half()
    b = torch.randn(20, 8, device="cuda").half()
    b[0, 0], b[1, 1] = -0.0, float("nan")
    y, t = ad(x, b, g)
    assert torch.equal(y.view(torch.int16), b.view(torch.int16)) and not bool(t.any())
    d = torch.randn(20, 16, device="cuda").half()
    dx, dA, dB = ad.backward(b, x, t, g, dx=d)
    assert torch.equal(dx, d) and not bool(dA.any()) and not bool(dB.any())
    dx, _, _ = ad.backward(b, x, t, g)
    assert not bool(dx.any())
    # adapter 1 has all rows
    g = group(np.full(20, 1), 3)
    x = torch.randn(20, 16, device="cuda").half()
    _, dA, dB = ad.backward(torch.randn(20, 8, device="cuda").half(), x, torch.randn(20, 4, device="cuda"), g)
    for d in (dA, dB):
        assert not bool(d[0].any()) and not bool(d[2].any()) and bool(d[1].all())


@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_rows_and_groups_do_not_meet(gpu, name):
    """A row's NaN stays in its row, in its adapter's gradients and out of the others'."""
    torch = _torch()
    rng = np.random.default_rng(31)
    rows, count, n, m, rank = 80, 4, 64, 96, 16
    index = rng.integers(0, count, rows)
    g = group(index, count)
    x, _ = to_dev(rng.standard_normal((rows, m)), name)
    base, _ = to_dev(rng.standard_normal((rows, n)), name)
    A, _ = to_dev(rng.standard_normal((count, rank, m)), name)
    B, _ = to_dev(rng.standard_normal((count, n, rank)), name)
    ad = dbf.Adapters(A, B)
    y, t = ad(x, base, g)
    bad = x.clone()
    bad[7, 3] = float("nan")
    yb, tb = ad(bad, base, g)
    keep = [r for r in range(rows) if r != 7]
    assert torch.equal(y[keep], yb[keep]) and torch.equal(t[keep], tb[keep])
    assert bool(yb[7].isnan().all()) and bool(tb[7].isnan().all())
    dy, _ = to_dev(rng.standard_normal((rows, n)), name)
    dx, dA, dB = ad.backward(dy, x, t, g)
    dxb, dAb, dBb = ad.backward(dy, bad, tb, g)
    others = [a for a in range(count) if a != index[7]]
    assert torch.equal(dx, dxb)
    assert torch.equal(dA[others], dAb[others]) and torch.equal(dB[others], dBb[others])
    assert bool(dAb[index[7], :, 3].isnan().all()) and bool(dBb[index[7]].isnan().all())


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rank", [3, 8, 16, 20, 40, 100])
@pytest.mark.parametrize("rows", [4, 600])
def test_infinities(gpu, rows, rank, name):
    """An infinite x is what it is in the formula: infinities of the products' signs, NaN only where they meet."""
    torch = _torch()
    rng = np.random.default_rng(rank)
    n, m = 72, 9000 if rows == 600 else 136
    x, _ = to_dev(rng.uniform(0.5, 1, (rows, m)), name)
    x[1, 5], x[2, 7] = float("inf"), float("-inf")
    A, _ = to_dev(rng.uniform(0.5, 1, (1, rank, m)), name)
    B = rng.uniform(0.5, 1, (1, n, rank)) * np.where(rng.random((1, n, 1)) < 0.5, -1, 1)
    B[0, 0, 0] *= -1  # both signs in one sum: NaN
    B, _ = to_dev(B, name)
    base = torch.zeros(rows, n, dtype=T(name), device="cuda")
    g = group(np.zeros(rows, int), 1)
    y, t = dbf.Adapters(A, B)(x, base, g)
    low = x.double() @ A[0].double().t()
    ref = low @ B[0].double().t()
    assert torch.equal(torch.nan_to_num(t, 0, 1, -1)[1:3], torch.nan_to_num(low, 0, 1, -1).float()[1:3])
    assert torch.equal(y[1:3].isnan(), ref[1:3].isnan()) and bool(ref[1, 0].isnan())
    assert torch.equal(torch.nan_to_num(y, 0, 1, -1)[1:3], torch.nan_to_num(ref, 0, 1, -1).to(T(name))[1:3])
    dy = torch.zeros(rows, n, dtype=T(name), device="cuda")
    dy[:] = B[0, :, 0]
    dy[1, 3] = float("inf")
    dx, _, _ = dbf.Adapters(A, B.abs()).backward(dy, x, torch.ones(rows, rank, device="cuda"), g)
    assert bool((dx[1] == float("inf")).all()) and bool(torch.isfinite(dx[3].float()).all())


def test_large_and_small_magnitudes(gpu):
    """f16 values whose t is far outside of f16's range, and gradients far below it."""
    torch = _torch()
    rng = np.random.default_rng(41)
    rows, n, m, rank = 20, 48, 512, 8
    index = np.zeros(rows, int)
    g = group(index, 1)
    x, xv = to_dev(rng.uniform(500, 1000, (rows, m)), "f16")
    A, Av = to_dev(rng.uniform(100, 1000, (1, rank, m)), "f16")
    B, Bv = to_dev(rng.uniform(0.5, 1, (1, n, rank)) * 2.0 ** -18, "f16")
    base = torch.zeros(rows, n, device="cuda").half()
    y, t = dbf.Adapters(A, B)(x, base, g)
    yr, tr = O.adapters(xv, np.zeros((rows, n)), Av, Bv, np.ones(1), index)
    assert np.abs(tr).max() > 1e8 and np.abs(yr).max() < 65504  # t of more than f16 holds
    within(t.double().cpu().numpy(), tr, (m / 8 + 16) * 2.0 ** -24 * tr, "t")
    within(y.double().cpu().numpy(), yr, (2.0 ** -11 + (m / 8 + rank / 4 + 40) * 2.0 ** -23) * yr, "y")
    dy, dyv = to_dev(rng.uniform(1, 2, (rows, n)) * 2.0 ** -20, "f16")
    small, sv = to_dev(rng.uniform(0.5, 1, (1, n, rank)) * 2.0 ** -20, "f16")
    _, dA, _ = dbf.Adapters(A, small).backward(dy, x, t, g)
    _, _, dAr, _ = O.adapters_backward(dyv, xv, tr, np.zeros((rows, m)), Av, sv, np.ones(1), index)
    within(dA.double().cpu().numpy(), dAr, (n / 8 + 3 * rows / 8 + 60) * 2.0 ** -23 * dAr, "dA")


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
@pytest.mark.parametrize("rows", [130, 2500])
def test_rows_of_changing_magnitude(gpu, rows, order, name):
    """dB of rows whose t goes from 0 and 2^-40 to 2^40: each wave's power of two follows the rows, in any order."""
    _say(f"adapters: {rows} rows, t {order}, {name}")
    torch = _torch()
    rng = np.random.default_rng(rows)
    count, n, m, rank = 2, 72, 40, 20
    index = np.sort(rng.integers(0, count, rows))
    power = np.linspace(-40, 40, rows)
    power = power[::-1] if order == "falling" else rng.permutation(power) if order == "mixed" else power
    tv = (rng.standard_normal((rows, rank)) * 2.0 ** power[:, None]).astype(np.float32)
    tv[:40] = 0
    dy, dyv = to_dev(rng.standard_normal((rows, n)), name)
    x, _ = to_dev(rng.standard_normal((rows, m)), name)
    A, _ = to_dev(rng.standard_normal((count, rank, m)), name)
    B, _ = to_dev(rng.standard_normal((count, n, rank)), name)
    _, _, dB = dbf.Adapters(A, B).backward(dy, x, torch.from_numpy(tv).cuda(), group(index, count))
    v = tv.astype(np.float64)
    loose = parts_error(v, index, name, True) + (3 * rows / 8 + 20) * 2.0 ** -24 * np.abs(v)
    for a in range(count):
        at = index == a
        ref, tol = dyv[at].T @ v[at], np.abs(dyv[at]).T @ loose[at]
        within(dB[a].double().cpu().numpy(), ref, tol + 2.0 ** -149, f"dB of {a}")


def test_nothing_outside_the_results(gpu):
    torch = _torch()
    rng = np.random.default_rng(51)
    for n, m, rank in ((40, 64, 16), (37, 61, 5)):
        rows, count = 50, 3
        g = group(spread(rng, rows, count), count)
        A, B = torch.randn(count, rank, m, device="cuda").half(), torch.randn(count, n, rank, device="cuda").half()
        ad = dbf.Adapters(A, B)
        x, base = torch.randn(rows, m, device="cuda").half(), torch.randn(rows, n, device="cuda").half()
        room = torch.full((32 + rows * n,), 7.0, device="cuda").half()
        out = room[16:16 + rows * n].view(rows, n)
        y, t = ad(x, base, g, out=out)
        assert torch.equal(out, ad(x, base, g).y)
        assert bool((room[:16] == 7).all()) and bool((room[16 + rows * n:] == 7).all())
        room = torch.full((32 + rows * m,), 7.0, device="cuda").half()
        out = room[16:16 + rows * m].view(rows, m)
        ad.backward(base, x, t, g, out=out)
        assert bool((room[:16] == 7).all()) and bool((room[16 + rows * m:] == 7).all())
        # orders of other origin: inside the buffers
        order = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, rows)).to(torch.int32).cuda()
        for offsets in ([0, rows, 0, rows], [-5, 1000, 2 ** 31 - 1, -2 ** 31], [rows, 30, 20, 10]):
            h = dbf.RowGroups(order, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
            room.fill_(7.0)
            ad(x, base, h)
            ad.backward(base, x, t, h, out=out)
            torch.cuda.synchronize()
            assert bool((room[:16] == 7).all()) and bool((room[16 + rows * m:] == 7).all())


def test_partial_gradients_by_the_c_entry(gpu):
    """Each of dx', dA and dB alone is what it is together with the others."""
    torch = _torch()
    rng = np.random.default_rng(61)
    rows, count, n, m, rank = 700, 2, 64, 128, 16
    g = group(spread(rng, rows, count), count)
    x, dy = torch.randn(rows, m, device="cuda").bfloat16(), torch.randn(rows, n, device="cuda").bfloat16()
    t = torch.randn(rows, rank, device="cuda")
    ad = dbf.Adapters(torch.randn(count, rank, m, device="cuda").bfloat16(),
                      torch.randn(count, n, rank, device="cuda").bfloat16())
    want = ad.backward(dy, x, t, g)
    L = dbf.lib()
    nbytes = L.dbf_adapter_backward_workspace(rows, n, m, rank, count)
    for k in range(3):
        ws = torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")  # NaN in every type
        got = torch.empty_like(want[k])
        ptr = [got.data_ptr() if i == k else None for i in range(3)]
        assert L.dbf_adapter_backward(dy.data_ptr(), x.data_ptr(), t.data_ptr(), None, ad.A.data_ptr(), ad.B.data_ptr(),
                                      None, dbf.DBF_TYPE_BF16, g.order.data_ptr(), g.offsets.data_ptr(), rows, n, m, rank,
                                      count, *ptr, ws.data_ptr(), nbytes, torch.cuda.current_stream().cuda_stream) == 0
        assert torch.equal(got, want[k])


def test_captured_replays(gpu):
    """Forward and backward in one graph, replayed on new rows and indexes, with eager work between."""
    torch = _torch()
    rng = np.random.default_rng(71)
    rows, count, n, m, rank = 150, 3, 96, 128, 16
    x, base = torch.zeros(rows, m, device="cuda").bfloat16(), torch.zeros(rows, n, device="cuda").bfloat16()
    dy = torch.zeros(rows, n, device="cuda").bfloat16()
    index = torch.zeros(rows, dtype=torch.int32, device="cuda")
    ad = dbf.Adapters(torch.randn(count, rank, m, device="cuda").bfloat16(),
                      torch.randn(count, n, rank, device="cuda").bfloat16())

    def step():
        g = dbf.group_rows(index, count)
        y, t = ad(x, base, g)
        return (y, t) + ad.backward(dy, x, t, g)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(4):
        r = np.random.default_rng(seed)
        index.copy_(torch.from_numpy(spread(r, rows, count)).to(torch.int32))
        for v in (x, base, dy):
            v.copy_(torch.from_numpy(r.standard_normal(tuple(v.shape))).bfloat16())
        graph.replay()
        held = [v.clone() for v in got]
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)


def test_refusals(gpu):
    torch = _torch()
    A, B = torch.randn(3, 4, 16, device="cuda").half(), torch.randn(3, 8, 4, device="cuda").half()
    s = torch.ones(3, device="cuda")
    for bad in ((A[:2], B), (A, B.bfloat16()), (A.float(), B.float()), (A, B.transpose(1, 2)), (A, B, s.half()),
                (A, B, s[:2]), (A, B.cpu()), (A[:, :0], B[:, :, :0]), (A[0], B[0])):
        with pytest.raises(ValueError):
            dbf.Adapters(*bad)
    ad = dbf.Adapters(A, B, s)
    x, base, t = torch.randn(5, 16, device="cuda").half(), torch.randn(5, 8, device="cuda").half(), torch.zeros(5, 4, device="cuda")
    g, g4, g6 = group([0, 1, 2, 0, -1], 3), group([0, 1, 2, 0, -1], 4), group([0] * 6, 3)
    for call in (lambda: ad(x.bfloat16(), base, g), lambda: ad(x, base[:4], g), lambda: ad(base, base, g),
                 lambda: ad(x, x, g), lambda: ad(x, base, g4), lambda: ad(x, base, g6), lambda: ad(x, base, None),
                 lambda: ad(x, base, g, out=x), lambda: ad(x.t().contiguous().t(), base, g),
                 lambda: ad.backward(base, x, t.half(), g), lambda: ad.backward(base, x, t[:4], g),
                 lambda: ad.backward(x, x, t, g), lambda: ad.backward(base, base, t, g),
                 lambda: ad.backward(base, x, t, g, dx=base), lambda: ad.backward(base, x, t, g, out=base),
                 lambda: ad.backward(base, x, t, g6)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(dbf.DbfError):
        big = dbf.Adapters(torch.zeros(1, 129, 16, device="cuda").half(), torch.zeros(1, 8, 129, device="cuda").half())
        big(x, base, group([0] * 5, 1))
