"""GPU: products of 4-bit experts and their input gradients, against the fp64 oracle.

* on small whole numbers, where every sum is exact: bit for bit;
* on normal data: per output half a step of its type plus an accumulation
  term.  fp32 sums of K products: 2^-24 of Σ|a b| per addition, at most K / 32
  additions in a row (the matrix core adds 32 or more products at once), and
  for e4m3 rows what the matrix core cuts off: of eight consecutive columns
  less than 7 * 2^-13 of their largest product.

Every case prints its name before it touches the GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as M
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
    """Half of the type's smallest subnormal step."""
    return {"f16": 2.0 ** -25, "bf16": 2.0 ** -134}[name]


def to_dev(x, name):
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).to(T(name))
    return t.cuda(), t.double().numpy()


def blocks_to_dev(codes, scales, cols, fmt):
    torch = _torch()
    c, s = M.pad_rows(codes, scales, fmt)
    return dbf.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), cols, fmt)


def make(rng, count, n, m, max_rows, act="e4m3", whole=False):
    """(Experts, the weights' values)."""
    w = rng.integers(-3, 4, size=(count * n, m)).astype(float) if whole else rng.standard_normal((count * n, m)) * 0.02
    codes, s = M.quantize(w, "e2m1")
    v = M.values(codes, s, "e2m1")
    if whole:
        assert np.array_equal(v, w)
    W = blocks_to_dev(codes, s, m, "e2m1")
    return dbf.Experts(W, count, max_rows, act=act), [v[e * n:(e + 1) * n] for e in range(count)]


def group(index, count):
    torch = _torch()
    return dbf.group_rows(torch.from_numpy(np.asarray(index)).to(torch.int32).cuda(), count), O.group_rows(index, count)


def spread(rng, rows, count, none=0.1):
    """An uneven index: one popular group, some rows of none."""
    v = np.where(rng.random(rows) < 0.4, rng.integers(0, count), rng.integers(0, count, rows))
    return np.where(rng.random(rows) < none, -1, v)


def cut(xv, w):
    """Per output, the sum over eight columns of their largest product."""
    k = -(-xv.shape[1] // 8) * 8
    px, pw = np.zeros((xv.shape[0], k)), np.zeros((w.shape[0], k))
    px[:, :xv.shape[1]], pw[:, :w.shape[1]] = np.abs(xv), np.abs(w)
    out = np.zeros((xv.shape[0], w.shape[0]))
    for b in range(k // 8):
        out += np.max(px[:, None, 8 * b:8 * b + 8] * pw[None, :, 8 * b:8 * b + 8], axis=2)
    return out


def check(got, ref, mag, K, name, lost=0.0):
    y = got.double().cpu().numpy()
    acc = (K / 32 + 2) * 2.0 ** -24 * mag + lost
    tol = _torch().finfo(T(name)).eps / 2 * (np.abs(ref) + acc) + acc + tiny(name)
    d = np.abs(y - ref)
    assert np.all(d <= tol), f"worst {float((d / np.maximum(tol, 1e-300)).max()):.3f} of the tolerance"


SIZES = [  # count, n, m, tokens, top
    (1, 32, 32, 1, 1), (3, 33, 40, 2, 2), (8, 64, 128, 1, 2), (4, 100, 257, 17, 3), (13, 200, 300, 60, 4),
    (64, 48, 160, 16, 8), (2, 96, 4100, 40, 1), (5, 300, 128, 700, 2), (1024, 8, 32, 50, 3),
]


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("count,n,m,tokens,top", SIZES)
def test_forward_bits_on_whole_numbers(gpu, count, n, m, tokens, top, act, name):
    _say(f"experts bits {count}x{n}x{m} tokens {tokens} top {top} {act} {name}")
    rng = np.random.default_rng(count + n + m)
    ex, w = make(rng, count, n, m, tokens * top, act, whole=True)
    g, (order, offsets) = group(spread(rng, tokens * top, count), count)
    for gather, rows in ((top, tokens), (1, tokens * top), (0, tokens * top)):
        # e2m1 holds 0..4 and 6 (a block's scale is 1: a 4 in each); sums stay small
        x = rng.choice([-4.0, -2.0, -1.0, 0.0, 1.0, 2.0, 4.0], size=(rows, m))
        x[:, ::32] = 4.0
        xd, xv = to_dev(x, name)
        for scatter in (False, True):
            y = ex(xd, g, gather=gather, scatter=scatter)
            ref = O.experts(xv, w, order, offsets, gather, scatter)
            want = _torch().from_numpy(ref).to(T(name))
            assert _torch().equal(y.cpu(), want)
            q = dbf.mx_quantize(xd, act)
            assert _torch().equal(ex.forward(q, g, gather=gather, scatter=scatter, out_dtype=T(name)).cpu(), want)
    ex.close()


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("count,n,m,tokens,top", SIZES)
def test_forward(gpu, count, n, m, tokens, top, act, name):
    _say(f"experts {count}x{n}x{m} tokens {tokens} top {top} {act} {name}")
    rng = np.random.default_rng(7 * count + n + m)
    ex, w = make(rng, count, n, m, tokens * top, act)
    g, (order, offsets) = group(spread(rng, tokens * top, count), count)
    x = rng.standard_normal((tokens, m))
    x[:, rng.random(m) < 0.02] *= 20.0
    xd, xv = to_dev(x, name)
    y = ex(xd, g, gather=top)
    xq = M.values(*M.quantize(xv, act), act)
    ref = O.experts(xq, w, order, offsets, top, False)
    mag = O.experts(np.abs(xq), [np.abs(v) for v in w], order, offsets, top, False)
    lost = 0.0
    if act == "e4m3":
        lost = np.zeros_like(ref)
        for at, e in enumerate(O.places(order, offsets)):
            if e < count:
                lost[at] = 7 * 2.0 ** -13 * cut(xq[order[at] // top][None], w[e])[0]
    check(y, ref, mag, m, name, lost)
    ex.close()


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("count,n,m,tokens,top", SIZES + [(3, 1000, 64, 300, 2), (2, 513, 96, 33, 1)])
def test_backward(gpu, count, n, m, tokens, top, name):
    _say(f"experts backward {count}x{n}x{m} tokens {tokens} top {top} {name}")
    rng = np.random.default_rng(11 * count + n + m)
    slots = tokens * top
    g, (order, offsets) = group(spread(rng, slots, count), count)
    # whole numbers: bit for bit, in every order
    ex, w = make(rng, count, n, m, slots, whole=True)
    wt = [v.T for v in w]
    for gather, rows in ((0, slots), (1, slots), (top, tokens)):
        dyd, dyv = to_dev(rng.integers(-2, 3, size=(rows, n)), name)
        for scatter in (False, True):
            dx = ex.backward_data(dyd, g, gather=gather, scatter=scatter)
            ref = O.experts(dyv, wt, order, offsets, gather, scatter)
            assert _torch().equal(dx.cpu(), _torch().from_numpy(ref).to(T(name)))
    ex.close()
    ex, w = make(rng, count, n, m, slots)
    wt = [v.T for v in w]
    dyd, dyv = to_dev(rng.standard_normal((slots, n)) * 0.01, name)
    ref = O.experts(dyv, wt, order, offsets, 0, True)
    mag = O.experts(np.abs(dyv), [np.abs(v) for v in wt], order, offsets, 0, True)
    check(ex.backward_data(dyd, g, scatter=True), ref, mag, n, name)
    ex.close()


def test_every_tile(gpu):
    """Slots from one to thousands over few and many groups reach every tile of both products, with K whole and in
    parts: bit for bit on whole numbers."""
    torch = _torch()
    rng = np.random.default_rng(2)
    for count, n, m, slots in ((2, 256, 2048, 1), (2, 256, 2048, 40), (2, 512, 512, 200), (2, 2048, 256, 600),
                               (1, 2048, 1024, 2300), (2, 64, 8192, 5)):
        _say(f"every tile {count} x {n} x {m}, {slots} slots")
        ex, w = make(rng, count, n, m, slots, whole=True)
        wd = [torch.from_numpy(v).float().cuda() for v in w]
        index = rng.integers(0, count, slots)
        g, (order, offsets) = group(index, count)
        for name in ("f16", "bf16"):
            x = torch.from_numpy(rng.integers(-1, 2, size=(slots, m))).to(T(name)).cuda()
            dy = torch.from_numpy(rng.integers(-1, 2, size=(slots, n))).to(T(name)).cuda()
            y, dx = ex(x, g), ex.backward_data(dy, g)
            q = dbf.mx_quantize(x, "e2m1")
            y4 = ex.forward(q, g, out_dtype=T(name))
            for e in range(count):
                s = slice(offsets[e], offsets[e + 1])
                ref = (x[s].float() @ wd[e].t()).to(T(name))  # whole numbers below 2^24: exact in fp32
                assert torch.equal(y[s], ref) and torch.equal(y4[s], ref)
                assert torch.equal(dx[s], (dy[s].float() @ wd[e]).to(T(name)))
        ex.close()


def test_no_rows_and_none_of_any_group(gpu):
    torch = _torch()
    rng = np.random.default_rng(1)
    ex, _ = make(rng, 3, 40, 64, 50)
    empty = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    g = dbf.group_rows(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert ex(empty, g).shape == (0, 40) and ex.backward_data(empty.new_empty(0, 40), g).shape == (0, 64)
    g, _ = group(np.full(50, -1), 3)
    x = torch.full((50, 64), float("nan"), dtype=torch.float16, device="cuda")
    for scatter in (False, True):
        assert torch.equal(ex(x, g, scatter=scatter), torch.zeros(50, 40, dtype=torch.float16, device="cuda"))
        assert torch.equal(ex.backward_data(torch.full((50, 40), float("inf"), dtype=torch.float16, device="cuda"), g,
                                            scatter=scatter), torch.zeros(50, 64, dtype=torch.float16, device="cuda"))
    ex.close()


def test_rows_do_not_meet(gpu):
    """NaN and infinite rows leave the others' bits alone, and so do the rows beside a row."""
    torch = _torch()
    rng = np.random.default_rng(9)
    ex, _ = make(rng, 4, 96, 256, 64)
    index = rng.integers(0, 4, 64)
    g, (order, _) = group(index, 4)
    x = torch.from_numpy(rng.standard_normal((64, 256))).to(torch.bfloat16).cuda()
    y = ex(x, g, gather=1, scatter=True)
    bad = x.clone()
    bad[5, 7], bad[20, 0] = float("nan"), float("inf")
    yb = ex(bad, g, gather=1, scatter=True)
    keep = [r for r in range(64) if r not in (5, 20)]
    assert torch.equal(y[keep], yb[keep]) and bool(yb[5].isnan().all()) and bool(yb[20].isnan().all())
    dy = torch.from_numpy(rng.standard_normal((64, 96))).to(torch.bfloat16).cuda()
    dx = ex.backward_data(dy, g, gather=1, scatter=True)
    dy[9, 3] = float("nan")
    dxb = ex.backward_data(dy, g, gather=1, scatter=True)
    keep = [r for r in range(64) if r != 9]
    assert torch.equal(dx[keep], dxb[keep]) and bool(dxb[9].isnan().all())
    ex.close()


def test_nothing_outside_the_result(gpu):
    torch = _torch()
    rng = np.random.default_rng(4)
    for n in (40, 37):
        ex, _ = make(rng, 3, n, 64, 77)
        g, _ = group(spread(rng, 77, 3), 3)
        x = torch.randn(77, 64, device="cuda", dtype=torch.float16)
        for scatter in (False, True):
            room = torch.full((2 * 16 + 77 * n,), 7.0, dtype=torch.float16, device="cuda")
            out = room[16:16 + 77 * n].view(77, n)
            ex.forward(x, g, scatter=scatter, out=out)
            assert bool((room[:16] == 7).all()) and bool((room[16 + 77 * n:] == 7).all())
            assert torch.equal(out, ex(x, g, scatter=scatter))
        ex.close()


def test_orders_of_other_origin_stay_inside(gpu):
    """Places and offsets out of range: rows clamped or left out, nothing outside the buffers."""
    torch = _torch()
    rng = np.random.default_rng(6)
    ex, _ = make(rng, 3, 40, 64, 60)
    room = torch.full((32 + 60 * 40,), 7.0, dtype=torch.float16, device="cuda")
    out = room[16:16 + 60 * 40].view(60, 40)
    x = torch.randn(60, 64, device="cuda", dtype=torch.float16)
    for offsets in ([0, 60, 0, 60], [-5, 1000, 2 ** 31 - 1, -2 ** 31], [60, 50, 40, 30]):
        order = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, 60)).to(torch.int32).cuda()
        g = dbf.RowGroups(order, torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        for gather, scatter in ((0, True), (2, False), (1, True)):
            ex.forward(x[:30] if gather == 2 else x, g, gather=gather, scatter=scatter, out=out)
    torch.cuda.synchronize()
    assert bool((room[:16] == 7).all()) and bool((room[16 + 60 * 40:] == 7).all())
    ex.close()


def test_captured_replays(gpu):
    """A captured pass (sorting, up, down) follows its inputs; eager work between the replays."""
    torch = _torch()
    rng = np.random.default_rng(8)
    tokens, top, count = 33, 2, 5
    up, _ = make(rng, count, 192, 128, tokens * top)
    down, _ = make(rng, count, 128, 192, tokens * top)
    index = torch.zeros(tokens * top, dtype=torch.int32, device="cuda")
    x = torch.zeros(tokens, 128, dtype=torch.bfloat16, device="cuda")

    def step():
        g = dbf.group_rows(index, count)
        return down(up(x, g, gather=top), g, scatter=True)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step()
    for seed in range(4):
        r = np.random.default_rng(seed)
        index.copy_(torch.from_numpy(spread(r, tokens * top, count)).to(torch.int32))
        x.copy_(torch.from_numpy(r.standard_normal((tokens, 128))).to(torch.bfloat16))
        graph.replay()
        got = y.clone()
        torch.cuda.synchronize()
        assert torch.equal(got, step())
    up.close()
    down.close()


def test_other_stream_timing_info_and_refusals(gpu):
    torch = _torch()
    rng = np.random.default_rng(12)
    ex, _ = make(rng, 3, 40, 64, 12)
    x = torch.randn(12, 64, device="cuda", dtype=torch.float16)
    g, _ = group(rng.integers(0, 3, 12), 3)
    y = ex(x, g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        z = ex(x, g)
    side.synchronize()
    assert torch.equal(y, z)
    info = ex.info()
    assert info["n"] == 40 and info["m"] == 64 and info["max_batch"] == 12
    dbf.dbf_timing_enable(ex.handle)
    ex(x, g)
    assert {"mx_quantize", "mx_product"} <= set(dbf.dbf_timing_read(ex.handle))
    dbf.dbf_timing_enable(ex.handle, False)

    wide = torch.randn(12, 65, device="cuda", dtype=torch.float16)
    other, _ = group(rng.integers(0, 4, 12), 4)
    many, _ = group(rng.integers(0, 3, 13), 3)
    for call in (lambda: ex(wide, g), lambda: ex(x.float(), g), lambda: ex(x[:11], g), lambda: ex(x, other),
                 lambda: ex(torch.randn(13, 64, device="cuda").half(), many), lambda: ex(x, g, gather=2),
                 lambda: ex(x, g, gather=-1), lambda: ex(x[:5], g, gather=2), lambda: ex(x, (g.order, g.offsets)),
                 lambda: ex(x, g, out=x), lambda: ex(x, g, out_dtype=torch.float32), lambda: ex(x.t(), g),
                 lambda: ex.backward_data(x, g), lambda: ex.backward_data(y.float(), g),
                 lambda: ex.backward_data(y, g, out=y), lambda: ex.backward_data(y[:3], g)):
        with pytest.raises(ValueError):
            call()
    W = dbf.mx_quantize(torch.randn(12, 64, device="cuda"), "e2m1")
    for bad in ((W, 5, 4), (W, 0, 4), (dbf.mx_quantize(torch.randn(12, 64, device="cuda"), "e4m3"), 3, 4)):
        with pytest.raises(ValueError):
            dbf.Experts(*bad)
    # the other entry points do not take the handle
    L, p = dbf.lib(), x.data_ptr()
    import ctypes
    hs = (ctypes.c_void_p * 1)(ex.handle)
    ys = (ctypes.c_void_p * 1)(y.data_ptr())
    no = dbf.DBF_ERR_UNSUPPORTED
    assert L.dbf_linear_forward(ex.handle, p, y.data_ptr(), 1, None) == no
    assert L.dbf_linear_forward_noalloc(ex.handle, p, y.data_ptr(), 1, None) == no
    assert L.dbf_linear_forward_group(hs, 1, p, ys, 1, None) == no
    assert L.dbf_linear_backward_data(ex.handle, y.data_ptr(), p, 1, None) == no
    assert L.dbf_linear_backward(ex.handle, p, y.data_ptr(), p, None, None, None, 1, None) == no
    assert L.dbf_mx_forward(ex.handle, p, 0, None, y.data_ptr(), 0, 1, None) == no
    assert L.dbf_mx_backward_data(ex.handle, y.data_ptr(), p, 0, 1, None) == no
    layer = dbf.Layer.mx(W, max_batch=4)
    assert L.dbf_experts_forward(layer.handle, p, 0, None, None, g.offsets.data_ptr(), 4, 0, 0, y.data_ptr(), 0, None) == no
    f = lambda slots=12, gather=0, scatter=0, order=g.order.data_ptr(), offsets=g.offsets.data_ptr(): \
        L.dbf_experts_forward(ex.handle, p, 0, None, order, offsets, slots, gather, scatter, y.data_ptr(), 0, None)  # noqa: E731
    bad = dbf.DBF_ERR_INVALID_ARG
    assert f(slots=13) == bad and f(slots=-1) == bad and f(gather=-1) == bad and f(gather=5) == bad
    assert f(scatter=2) == bad and f(offsets=None) == bad and f(scatter=1, order=None) == bad
    assert f(gather=2, order=None) == bad and f(order=None) == 0 and f(slots=0, offsets=None) == 0
    torch.cuda.synchronize()
    layer.close()
    ex.close()
