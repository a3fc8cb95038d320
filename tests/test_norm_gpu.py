"""GPU: root-mean-square norm with the residual's addition, and its gradient, against the fp64 oracle.

Tolerances, in units of the compared value: a row's sum of squares is a sum of
non-negative fp32 terms, at most 32 of a lane in a row, 6 over the wave and 16
over the waves: relative error at most 56 * 2^-24 < 2^-18, halved by the root;
with the root, the division and two products: below 2^-18.  (Where the joins
are in fp64 it is less.)  Then half a step of the output's type.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as O
from tests.test_mx_gpu import T, half_step, rows_of, same_bits, tiny, to_dev

pytestmark = pytest.mark.gpu

REL = 2.0 ** -18


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


# widths of every kernel variant (one wave to sixteen per row), odd ones, block tails
SIZES = [(1, 1), (3, 7), (5, 32), (2, 100), (9, 512), (4, 513), (1, 1000), (33, 1024), (6, 1032), (3, 2048),
         (2, 3001), (1, 4096), (17, 4097), (2, 8192), (3, 8200), (2, 16384), (2, 16385), (1, 32768), (700, 264)]


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(gpu, rows, cols, name):
    import torch
    _say(f"norm {rows}x{cols} {name}")
    rng = np.random.default_rng(rows * 31 + cols)
    x, xv = to_dev(rows_of(rng, rows, cols), name)
    r, rv = to_dev(rows_of(rng, rows, cols, 0.5), name)
    eps = 1e-5
    # the fp32 epsilon that the call takes
    e32 = float(np.float32(eps))
    for residual in (None, r):
        for wname in (None, name, "f32"):
            w, wv = (None, np.ones(cols)) if wname is None else to_dev(1 + 0.2 * rng.standard_normal(cols), wname)
            out = dbf.rms_norm(x, w, residual=residual, eps=eps)
            if residual is None:
                assert out.h is x
                h = xv
            else:
                h = torch.from_numpy(xv + rv).to(T(name)).double().numpy()
                assert np.array_equal(out.h.double().cpu().numpy(), h)
            ref, rstd = O.rms_norm(h, wv, e32)
            assert np.all(np.abs(out.rstd.double().cpu().numpy() - rstd) <= REL * rstd)
            d = np.abs(out.y.double().cpu().numpy() - ref)
            assert np.all(d <= (half_step(name) * (1 + REL) + REL) * np.abs(ref) + tiny(name))
            # in blocks: the codes of the fp32 values
            q = dbf.rms_norm(x, w, residual=residual, eps=eps, mx=True)
            assert q.y.shape == (rows, cols) and q.y.fmt == "e4m3"
            codes, s = O.unpad_rows(q.y.codes.cpu().numpy(), q.y.scales.cpu().numpy(), cols, "e4m3")
            pc, ps = O.pad_rows(codes, s, "e4m3")
            assert np.array_equal(pc, q.y.codes.cpu().numpy()) and np.array_equal(ps, q.y.scales.cpu().numpy())
            check_blocks(codes, s, ref)


def check_blocks(codes, s, ref):
    """Each block's scale is right for some value within REL of its largest, and each code for some value within
    REL of its own."""
    rows, cols = ref.shape
    lo_s = O.quantize(ref * (1 - REL), "e4m3")[1].astype(int)
    hi_s = O.quantize(ref * (1 + REL), "e4m3")[1].astype(int)
    s = s.astype(int)
    assert np.all((s >= lo_s) & (s <= hi_s))
    inv = np.exp2(127.0 - np.repeat(s, 32, axis=1)[:, :cols])
    a = np.abs(ref) * inv
    got = np.abs(O.code_values("e4m3")[codes])
    lo = O.code_values("e4m3")[O.nearest_code(a * (1 - REL), "e4m3")]
    hi = O.code_values("e4m3")[O.nearest_code(a * (1 + REL), "e4m3")]
    assert np.all((got >= lo) & (got <= hi))
    assert np.all((np.sign(ref) * O.code_values("e4m3")[codes] >= 0))


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", SIZES + [(1500, 96), (2100, 40)])
def test_backward(gpu, rows, cols, name):
    """dx: the row's mean is a sum of fp32 terms of either sign: its error is REL times the mean of their
    magnitudes.  dweight: fp32 sums over the rows, at most 16 + parts / 16 + rows / parts additions in a row."""
    import torch
    _say(f"norm backward {rows}x{cols} {name}")
    rng = np.random.default_rng(rows * 17 + cols)
    h, hv = to_dev(rows_of(rng, rows, cols), name)
    dy, dyv = to_dev(rows_of(rng, rows, cols, 0.1), name)
    dh, dhv = to_dev(rows_of(rng, rows, cols, 0.1), name)
    rstd = (1 / np.sqrt((hv * hv).mean(axis=1) + 1e-5)).astype(np.float32)
    rd = torch.from_numpy(rstd).cuda()
    rv = rstd.astype(np.float64)
    for wname in (None, name, "f32"):
        w, wv = (None, np.ones(cols)) if wname is None else to_dev(1 + 0.2 * rng.standard_normal(cols), wname)
        ref, dw = O.rms_norm_backward(dyv, hv, wv, rv)
        xh = hv * rv[:, None]
        g = np.abs(dyv * wv)
        part = rv[:, None] * (g + np.abs(xh) * (g * np.abs(xh)).mean(axis=1, keepdims=True))
        for up in (None, dh):
            want = ref if up is None else ref + dhv
            dx, dwg = dbf.rms_norm_backward(dy, h, w, rd, dh=up)
            err = REL * part + 2.0 ** -23 * np.abs(want)
            d = np.abs(dx.double().cpu().numpy() - want)
            assert np.all(d <= half_step(name) * (np.abs(want) + err) + err + tiny(name))
            mag = np.abs(dyv * xh).sum(axis=0)
            assert dwg.dtype == torch.float32
            n_add = 16 + 128 + rows / 256
            assert np.all(np.abs(dwg.double().cpu().numpy() - dw) <= (n_add + 3) * 2.0 ** -24 * mag + 1e-45)
        again = dbf.rms_norm_backward(dy, h, w, rd, dh=dh)
        assert same_bits(again[0], dx) and same_bits(again[1], dwg)


@pytest.mark.parametrize("rows,cols", [(16500, 120), (8300, 256), (4200, 512), (2100, 1000), (1100, 2048), (531, 4096),
                                       (300, 8192), (257, 16384)])
def test_backward_many_rows(gpu, rows, cols):
    """More rows than the workgroups hold at a time, the last step incomplete (fp64 on the GPU; the tolerances of
    test_backward).  dweight: a lane adds at most rows / 256 rows, then 6 joins and 4 + 16 additions of parts."""
    import torch
    _say(f"norm backward many rows {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(rows)
    h = torch.randn((rows, cols), generator=g, device="cuda").bfloat16()
    dy = (0.1 * torch.randn((rows, cols), generator=g, device="cuda")).bfloat16()
    dh = (0.1 * torch.randn((rows, cols), generator=g, device="cuda")).bfloat16()
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).bfloat16()
    rstd = (h.double().square().mean(dim=1) + 1e-5).rsqrt().float()
    dx, dw = dbf.rms_norm_backward(dy, h, w, rstd, dh=dh)
    r = rstd.double()[:, None]
    xh, gw = h.double() * r, dy.double() * w.double()
    want = r * (gw - xh * (gw * xh).mean(dim=1, keepdim=True)) + dh.double()
    part = r * (gw.abs() + xh.abs() * (gw * xh).abs().mean(dim=1, keepdim=True))
    err = REL * part + 2.0 ** -23 * want.abs()
    assert bool(((dx.double() - want).abs() <= half_step("bf16") * (want.abs() + err) + err + tiny("bf16")).all())
    mag = (dy.double() * xh).abs().sum(dim=0)
    bound = (rows / 256 + 26 + 3) * 2.0 ** -24 * mag
    assert bool(((dw.double() - (dy.double() * xh).sum(dim=0)).abs() <= bound).all())
    again = dbf.rms_norm_backward(dy, h, w, rstd, dh=dh)
    assert same_bits(again[0], dx) and same_bits(again[1], dw)


def test_gradient_against_differences(gpu):
    """Directional differences of the forward itself (bf16 rows of few bits, fp32 statistics)."""
    _say("norm differences")
    rng = np.random.default_rng(3)
    rows, cols = 4, 96
    h = rng.integers(-8, 9, size=(rows, cols)) / 4.0
    hd, hv = to_dev(h, "bf16")
    w, wv = to_dev(1 + rng.integers(-4, 5, size=cols) / 16.0, "bf16")
    dy, dyv = to_dev(rng.integers(-8, 9, size=(rows, cols)) / 8.0, "bf16")
    out = dbf.rms_norm(hd, w, eps=1e-5)
    dx, dw = dbf.rms_norm_backward(dy, hd, w, out.rstd)
    v = rng.standard_normal((rows, cols))
    d = 1e-4
    f = lambda s: (O.rms_norm(hv + s * v, wv, 1e-5)[0] * dyv).sum()  # noqa: E731
    num = (f(d) - f(-d)) / (2 * d)
    got = (dx.double().cpu().numpy() * v).sum()
    # bf16 rounding of dx: half a step per term
    assert abs(num - got) <= half_step("bf16") * (np.abs(dx.double().cpu().numpy()) * np.abs(v)).sum() * 1.01 + 1e-4
    u = rng.standard_normal(cols)
    num = ((O.rms_norm(hv, wv + u, 1e-5)[0] - O.rms_norm(hv, wv, 1e-5)[0]) * dyv).sum()
    assert abs(num - (dw.double().cpu().numpy() * u).sum()) <= 1e-4


def test_special_rows(gpu):
    """Rows of zeros, of the type's largest values, with a NaN, with an infinity; the rows beside them unchanged."""
    import torch
    _say("norm special rows")
    for name in ("f16", "bf16"):
        for cols in (40, 2048, 5000):
            rng = np.random.default_rng(cols)
            x, _ = to_dev(rng.standard_normal((6, cols)), name)
            plain = dbf.rms_norm(x, None, eps=1e-6)
            plain_q = dbf.rms_norm(x, None, eps=1e-6, mx=True)
            x[1] = 0
            x[2] = torch.finfo(T(name)).max
            x[3, cols // 2] = float("nan")
            x[4, cols - 1] = float("inf")
            out = dbf.rms_norm(x, None, eps=1e-6)
            q = dbf.rms_norm(x, None, eps=1e-6, mx=True)
            for i in (0, 5):
                assert torch.equal(out.y[i], plain.y[i])
                assert torch.equal(q.y.codes[i], plain_q.y.codes[i]) and torch.equal(q.y.scales[i], plain_q.y.scales[i])
            v = q.y.dequantize()
            assert bool((out.y[1] == 0).all()) and bool((v[1] == 0).all())
            if name == "f16":
                # 65504² * 5000 is inside fp32: every value 1; in blocks 1, or where fp32 has it just below a
                # power of two, and so the scale one lower, 448 * 2^-9
                assert bool((out.y[2] == 1).all()) and bool(((v[2] == 1) | (v[2] == 0.875)).all())
            else:              # the squares overflow: rstd 0
                assert bool((out.y[2] == 0).all()) and bool((v[2] == 0).all())
            assert bool(torch.isnan(out.y[3]).all()) and bool(torch.isnan(v[3]).all())
            assert bool(torch.isnan(out.y[4, cols - 1])) and bool((out.y[4, :cols - 1] == 0).all())
            last = (cols - 1) // 32 * 32
            assert bool(torch.isnan(v[4, last:]).all()) and bool((v[4, :last] == 0).all())


def test_in_place_and_no_rows(gpu):
    import torch
    _say("norm in place")
    rng = np.random.default_rng(4)
    x, _ = to_dev(rng.standard_normal((5, 1032)), "bf16")
    r, _ = to_dev(rng.standard_normal((5, 1032)), "bf16")
    want = dbf.rms_norm(x, None, residual=r)
    st = torch.cuda.current_stream().cuda_stream
    x2, r2 = x.clone(), r.clone()
    code = dbf.lib().dbf_rms_norm(x2.data_ptr(), r2.data_ptr(), None, 1, 1, 5, 1032, 1e-6, r2.data_ptr(),
                                  x2.data_ptr(), 1, None, None, st)
    assert code == dbf.DBF_OK
    assert same_bits(x2, want.y) and same_bits(r2, want.h)
    e = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    out = dbf.rms_norm(e, None, residual=e, mx=True)
    assert out.y.shape == (0, 64)
    dx, dw = dbf.rms_norm_backward(e, e, None, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_most_rows(gpu):
    """As many rows as the interface counts: row offsets past 32 bits, a rounded-up row count past 31."""
    import torch
    _say("norm 2^31 - 1 rows")
    rows = 2 ** 31 - 1
    x = torch.empty((rows, 1), dtype=torch.float16, device="cuda")
    x.fill_(2.0)
    x[-1] = -3.0
    x[rows // 2] = 0.0
    out = dbf.rms_norm(x, None, eps=0.25)
    for i, v in ((0, 2.0), (rows // 2, 0.0), (rows - 2, 2.0), (rows - 1, -3.0)):
        want = v / np.sqrt(v * v + 0.25)
        assert abs(float(out.y[i]) - want) <= abs(want) * (half_step("f16") * (1 + REL) + REL)
    dx, dw = dbf.rms_norm_backward(x, x, None, out.rstd)
    # dy = h: dx = r (h - h r² h²) and Σ dy h r, all terms equal but two
    r = 1 / np.sqrt(4.25)
    want = r * (2 - 2 * r * r * 4)
    assert abs(float(dx[0]) - want) <= half_step("f16") * abs(want) * (1 + REL) + 8 * REL
    total = (rows - 2) * 4 * r + 9 / np.sqrt(9.25)
    # a lane adds 2^31 / 2^14 terms that all round alike: half a step of its sum each time at worst
    assert abs(float(dw[0]) - total) <= total * 2 ** 17 * 2.0 ** -24


def test_more_rows_than_a_launch(gpu):
    """Rows past one launch's, residual and blocks too: the bits of a small call on the same rows."""
    import torch
    _say("norm several launches")
    rows, cols = 2 ** 25 + 100, 40
    x = torch.randn((rows, cols), device="cuda").half()
    r = torch.randn((rows, cols), device="cuda").half()
    w = torch.randn(cols, device="cuda").half()
    for mx in (False, True):
        out = dbf.rms_norm(x, w, residual=r, mx=mx)
        for part in (slice(0, 64), slice(2 ** 25 - 64, 2 ** 25 + 64), slice(rows - 32, rows)):
            want = dbf.rms_norm(x[part].clone(), w, residual=r[part].clone(), mx=mx)
            assert torch.equal(out.h[part], want.h) and torch.equal(out.rstd[part], want.rstd)
            if mx:
                assert torch.equal(out.y.codes[part], want.y.codes) and torch.equal(out.y.scales[part], want.y.scales)
            else:
                assert torch.equal(out.y[part], want.y)


def test_feeds_a_sign_layer(gpu):
    """The 16-bit output in front of a sign-factor layer, as a decoder block runs it."""
    import torch
    from oracle import dbf_oracle
    from tests import inputs
    _say("norm into a sign layer")
    R = inputs.random_layer("norm feed", 128, 256, 192, 0, 0.05, 0.05, 0.05, (3,))
    L = dbf.Layer(R.A, R.B, R.a, R.mid, R.b, max_batch=3)
    try:
        x, _ = to_dev(np.random.default_rng(0).standard_normal((3, 256)), "f16")
        out = dbf.rms_norm(x, None, residual=x)
        y = L(out.y)
        torch.cuda.synchronize()
        ref = dbf_oracle.dense_forward(out.y.cpu().numpy(), R.A, R.B, R.a, R.mid, R.b)
        err = np.abs(y.double().cpu().numpy() - ref).max(axis=1) / np.abs(ref).max(axis=1)
        assert err.max() <= 2e-3
    finally:
        L.close()
