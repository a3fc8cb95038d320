"""GPU: block formats, layers with a 4-bit block weight, against the fp64 oracle.

* quantisation and the values: bit for bit (the scale is a power of two and
  each value is rounded once, so the oracle's result is the only right one);
* products on small whole numbers, where every sum is exact: bit for bit;
* products on normal data: per output half a step of its type plus an
  accumulation term times Σ|a b|.  fp32 sums of K products: 2^-24 per
  addition, at most K / 32 additions in a row (the matrix core adds 32 or
  more products at once).  e4m3 products are aligned with each other inside
  the matrix core; what falls below 2^-12 of the largest is lost, at most
  2^-12 of Σ|a b| in all;
* every call form of a layer (16-bit rows, ready blocks, grouped, without
  allocation, captured) gives the same bits.

Every case prints its name before it touches the GPU.
"""

import ctypes
import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as O
from tests import inputs

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def _torch():
    import torch
    return torch


def T(name):
    torch = _torch()
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def half_step(name):
    return _torch().finfo(T(name)).eps / 2


def tiny(name):
    """Half of the type's smallest subnormal step."""
    return {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}[name]


def rows_of(rng, rows, cols, scale=1.0):
    """Rows of normal values with a few large columns, a row of zeros among several."""
    x = rng.standard_normal((rows, cols)) * scale
    x[:, rng.random(cols) < 0.02] *= 20.0
    if rows > 2:
        x[rows // 2] = 0.0
    return x


def to_dev(x, name):
    """numpy values as a CUDA tensor of the type, and the values it holds in fp64."""
    torch = _torch()
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float64)).to(T(name))
    return t.cuda(), t.double().numpy()


def blocks_to_dev(codes, scales, cols, fmt):
    torch = _torch()
    c, s = O.pad_rows(codes, scales, fmt)
    return dbf.MxTensor(torch.from_numpy(c).cuda(), torch.from_numpy(s).cuda(), cols, fmt)


def weight(rng, n, m):
    """A weight in e2m1 blocks: (MxTensor, its fp64 values)."""
    codes, s = O.quantize(rng.standard_normal((n, m)) * 0.02, "e2m1")
    return blocks_to_dev(codes, s, m, "e2m1"), O.values(codes, s, "e2m1")


def same_bits(a, b):
    torch = _torch()
    v = torch.int16 if a.element_size() == 2 else torch.int32
    return torch.equal(a.view(v), b.view(v))


def check(y, ref, mag, K, name, exact_products):
    """|y - ref| within half a step of the type and the accumulation term."""
    y = y.double().cpu().numpy()
    acc = (K / 32 + 2) * 2.0 ** -24 + (0.0 if exact_products else 2.0 ** -12)
    tol = half_step(name) * (np.abs(ref) + acc * mag) + acc * mag + tiny(name)
    d = np.abs(y - ref)
    worst = float((d / np.maximum(tol, 1e-300)).max()) if d.size else 0.0
    assert np.all(d <= tol), f"worst {worst:.3f} of the tolerance"


# ---------------------------------------------------------------- the format

@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (5, 32), (2, 33), (7, 257), (1, 4096), (130, 1000), (33, 384)])
def test_quantize_bits(gpu, rows, cols, name, fmt):
    _say(f"quantize {rows}x{cols} {name} {fmt}")
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rows_of(rng, rows, cols) * np.exp2(rng.integers(-12, 6, size=(rows, 1)))
    xd, xv = to_dev(x, name)
    q = dbf.mx_quantize(xd, fmt)
    codes, s = O.quantize(xv, fmt)
    want_c, want_s = O.pad_rows(codes, s, fmt)  # the padding's zero bytes included
    got_c, got_s = q.codes.cpu().numpy(), q.scales.cpu().numpy()
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)
    for out in ("f32", "f16", "bf16"):
        v = q.dequantize(T(out)).cpu()
        want = _torch().from_numpy(O.values(codes, s, fmt)).to(T(out))
        assert _torch().equal(v, want), out


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("name", ["f16", "bf16", "f32"])
def test_quantize_every_magnitude(gpu, name, fmt):
    """Every bit pattern of a 16-bit type (fp32: random patterns, subnormals and the largest among them),
    neighbours in a block differing by up to 2^12; non-finite values make their block NaN."""
    torch = _torch()
    _say(f"quantize patterns {name} {fmt}")
    if name == "f32":
        rng = np.random.default_rng(7)
        bits = rng.integers(0, 1 << 32, size=1 << 16, dtype=np.uint64).astype(np.uint32)
        bits = np.sort(bits & np.uint32(0x7fffffff)) | (bits & np.uint32(0x80000000))
        bits[:64] = np.arange(64, dtype=np.uint32) * 1000003 % (1 << 23)
        bits[64:96] = 0x7f7fffff
        x = torch.from_numpy(bits.view(np.float32).copy())
    else:
        b = np.arange(1 << 16, dtype=np.uint16)
        x = torch.from_numpy(b.view(np.int16).copy()).view(T(name))
    x = x.reshape(-1, 256)
    q = dbf.mx_quantize(x.cuda(), fmt)
    xv = x.double().numpy()
    codes, s = O.quantize(xv, fmt)
    want_c, want_s = O.pad_rows(codes, s, fmt)
    assert np.array_equal(q.scales.cpu().numpy(), want_s)
    assert np.array_equal(q.codes.cpu().numpy(), want_c)
    v = q.dequantize(torch.float32).cpu().numpy()
    assert np.array_equal(v, O.values(codes, s, fmt).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_dequantize_every_code_and_scale(gpu, fmt):
    torch = _torch()
    _say(f"dequantize all {fmt}")
    ncode = 256 if fmt == "e4m3" else 16
    codes = np.tile(np.arange(ncode, dtype=np.uint8), 256 // ncode)[None, :].repeat(256, axis=0)
    scales = np.arange(256, dtype=np.uint8)[:, None].repeat(8, axis=1)
    q = blocks_to_dev(codes, scales, 256, fmt)
    want = torch.from_numpy(O.values(codes, scales, fmt))
    for out in ("f32", "f16", "bf16"):
        got = q.dequantize(T(out)).cpu().double().numpy()
        # (fp64 -> the type: torch rounds through fp32, which is exact for these values)
        assert np.array_equal(got, want.to(T(out)).double().numpy(), equal_nan=True), out


def test_more_rows_than_the_abi_counts(gpu):
    torch = _torch()
    _say("mx 2^31 rows refused")
    x = torch.empty((2 ** 31, 1), dtype=torch.float16, device="cuda")
    for call in (lambda: dbf.mx_quantize(x), lambda: dbf.rms_norm(x), lambda: dbf.rms_norm_backward(x, x, None, x)):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


def test_quantize_no_rows(gpu):
    torch = _torch()
    _say("quantize no rows")
    q = dbf.mx_quantize(torch.empty((0, 40), dtype=torch.float16, device="cuda"), "e2m1")
    assert q.shape == (0, 40) and q.dequantize().shape == (0, 40)


# ---------------------------------------------------------------- the product

SHAPES = [(1, 1, 1), (1, 16, 32), (2, 33, 31), (5, 100, 129), (16, 64, 512), (17, 65, 640), (31, 257, 1000),
          (64, 128, 256), (100, 300, 1300), (129, 1000, 260), (257, 520, 384), (300, 256, 2048)]


@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("b,n,m", SHAPES)
def test_forward(gpu, b, n, m, name, act):
    _say(f"mx forward b={b} n={n} m={m} {name} {act}")
    rng = np.random.default_rng(b * 7 + n * 3 + m)
    W, wv = weight(rng, n, m)
    xd, xv = to_dev(rows_of(rng, b, m), name)
    codes, s = O.quantize(xv, act)
    ref, mag = O.linear(O.values(codes, s, act), wv)
    L = dbf.Layer.mx(W, max_batch=b, act=act)
    try:
        y = L(xd)
        assert y.dtype == T(name)
        check(y, ref, mag, m, name, act == "e2m1")
        # ready blocks: the same bits
        y2 = L.forward(blocks_to_dev(codes, s, m, act), out_dtype=T(name))
        assert same_bits(y, y2)
    finally:
        L.close()


@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("b,n,m", [(1, 64, 512), (3, 100, 200), (16, 256, 1024), (40, 96, 160), (200, 300, 1500),
                                   (300, 520, 4096)])
def test_forward_whole_numbers(gpu, b, n, m, act):
    """Small whole numbers times powers of two: every product and sum is exact, so the bits are the oracle's."""
    _say(f"mx forward exact b={b} n={n} m={m} {act}")
    rng = np.random.default_rng(b + n + m)
    top = 4 if act == "e2m1" else 15
    x = rng.integers(-top, top + 1, size=(b, m)).astype(np.float64)
    x[x == 5] = 4
    if act == "e2m1":
        x[np.abs(x) == 5] = 4
    w = rng.integers(-4, 5, size=(n, m)).astype(np.float64)
    w[rng.random((n, m)) < 0.7] = 0
    wc, ws = O.quantize(w, "e2m1")
    xc, xs = O.quantize(x, act)
    xv, wv = O.values(xc, xs, act), O.values(wc, ws, "e2m1")
    # (15 / 16 * 512 = 480 saturates at 448: a block whose largest is 8..15 holds 15 as 14, a whole number still)
    assert np.array_equal(xv, np.round(xv))
    ref, mag = O.linear(xv, wv)
    assert mag.max() < 2 ** 24
    L = dbf.Layer.mx(blocks_to_dev(wc, ws, m, "e2m1"), max_batch=b, act=act)
    try:
        xd, _ = to_dev(x, "f16")
        for out in ("f16", "bf16"):
            y = L.forward(xd, out_dtype=T(out)).cpu()
            want = _torch().from_numpy(ref.astype(np.float32)).to(T(out))
            assert _torch().equal(y, want)
    finally:
        L.close()


def _device_products(a, b):
    """a @ bᵀ and |a| @ |b|ᵀ of fp64 numpy values, on the GPU in fp64 (sizes that take the CPU too long)."""
    torch = _torch()
    x, y = torch.from_numpy(a).cuda(), torch.from_numpy(np.ascontiguousarray(b.T)).cuda()
    return (x @ y).cpu().numpy(), (x.abs() @ y.abs()).cpu().numpy()


# every tile size, ragged in rows and columns, whole K and K in parts, K short of the pipeline's depth
LARGE = [(1900, 8100, 1030, "f16", "e4m3"), (1900, 8100, 1030, "bf16", "e2m1"), (1900, 4000, 1540, "bf16", "e4m3"),
         (1901, 4003, 1540, "f16", "e2m1"), (1000, 3990, 700, "f16", "e4m3"), (1000, 3990, 700, "bf16", "e2m1"),
         (300, 1000, 4100, "bf16", "e4m3"), (300, 1001, 4100, "f16", "e2m1"), (130, 500, 9000, "f16", "e4m3"),
         (1900, 8100, 100, "bf16", "e4m3"), (1900, 8100, 200, "f16", "e2m1"), (70, 60, 4096, "f16", "e2m1"), (400, 5001, 1030, "bf16", "e4m3"),
         (385, 3001, 1030, "f16", "e4m3"), (700, 2003, 700, "bf16", "e2m1"), (300, 2003, 1540, "f16", "e4m3"),
         (300, 2008, 1540, "bf16", "e2m1"), (300, 1001, 9000, "f16", "e4m3"), (250, 1001, 6000, "bf16", "e2m1"),
         (65, 1001, 4100, "f16", "e4m3"), (40, 1000, 4100, "bf16", "e2m1"), (17, 2001, 4096, "bf16", "e4m3"),
         (300, 1000, 14300, "bf16", "e4m3"), (400, 1000, 14300, "f16", "e2m1")]


@pytest.mark.parametrize("b,n,m,name,act", LARGE)
def test_forward_large(gpu, b, n, m, name, act):
    _say(f"mx forward large b={b} n={n} m={m} {name} {act}")
    rng = np.random.default_rng(b + n + m)
    W, wv = weight(rng, n, m)
    xd, xv = to_dev(rows_of(rng, b, m), name)
    codes, s = O.quantize(xv, act)
    ref, mag = _device_products(O.values(codes, s, act), wv)
    L = dbf.Layer.mx(W, max_batch=b, act=act)
    try:
        y = L(xd)
        check(y, ref, mag, m, name, act == "e2m1")
        for _ in range(3):
            assert same_bits(L(xd), y)
        assert same_bits(L.forward(blocks_to_dev(codes, s, m, act), out_dtype=T(name)), y)
    finally:
        L.close()


@pytest.mark.parametrize("act", ["e4m3", "e2m1"])
@pytest.mark.parametrize("b,n,m,name", [(16, 40, 8904, "f16"), (16, 40, 9216, "f16"), (13, 9001, 1100, "bf16"),
                                        (2, 9200, 4100, "f16"), (5, 33, 16384, "bf16"), (16, 33, 16376, "f16"),
                                        (3, 70, 16392, "bf16")])
def test_forward_few_rows(gpu, b, n, m, name, act):
    """Few rows at the widths where their blocks fill LDS, no longer fit it, or the sums change hands; several tiles
    of output rows for a workgroup; every run with the same bits."""
    _say(f"mx forward few rows b={b} n={n} m={m} {name} {act}")
    rng = np.random.default_rng(b + n + m)
    W, wv = weight(rng, n, m)
    xd, xv = to_dev(rows_of(rng, b, m), name)
    codes, s = O.quantize(xv, act)
    ref, mag = _device_products(O.values(codes, s, act), wv)
    L = dbf.Layer.mx(W, max_batch=b, act=act)
    try:
        y = L(xd)
        check(y, ref, mag, m, name, act == "e2m1")
        for _ in range(3):
            assert same_bits(L(xd), y)
        assert same_bits(L.forward(blocks_to_dev(codes, s, m, act), out_dtype=T(name)), y)
    finally:
        L.close()


def test_forward_batches_of_one_handle(gpu):
    """Every batch up to max_batch on one handle; a row's neighbours do not change it beyond the tolerance, and
    rows behind the batch stay as they were."""
    torch = _torch()
    _say("mx forward batches")
    rng = np.random.default_rng(11)
    n, m, top = 200, 700, 70
    W, wv = weight(rng, n, m)
    xd, xv = to_dev(rows_of(rng, top, m), "f16")
    codes, s = O.quantize(xv, "e4m3")
    ref, mag = O.linear(O.values(codes, s, "e4m3"), wv)
    L = dbf.Layer.mx(W, max_batch=top)
    try:
        for b in list(range(1, 20)) + [31, 32, 33, 48, 63, 64, 65, 70]:
            out = torch.full((top, n), 7.0, dtype=torch.float16, device="cuda")
            L.forward(xd[:b], out=out[:b])
            check(out[:b], ref[:b], mag[:b], m, "f16", False)
            assert bool((out[b:] == 7.0).all())
    finally:
        L.close()


@pytest.mark.parametrize("b", [1, 5, 40, 300])
def test_forward_nan_blocks(gpu, b):
    """A non-finite input value makes its own row NaN; a NaN scale of the weight its own output column."""
    torch = _torch()
    _say(f"mx nan b={b}")
    rng = np.random.default_rng(5)
    n, m = 70, 300
    codes, s = O.quantize(rng.standard_normal((n, m)), "e2m1")
    s[37, 2] = 255
    W = blocks_to_dev(codes, s, m, "e2m1")
    x = rng.standard_normal((b, m))
    x[b // 2, 299] = np.inf
    if b > 4:
        x[3, 0] = np.nan
    xd, _ = to_dev(x, "f16")
    L = dbf.Layer.mx(W, max_batch=b)
    try:
        y = L(xd).cpu().numpy()
        bad = np.zeros((b, n), bool)
        bad[b // 2] = True
        if b > 4:
            bad[3] = True
        bad[:, 37] = True
        assert np.array_equal(np.isnan(y), bad)
        assert np.isfinite(y[~bad]).all()
    finally:
        L.close()


def test_extreme_scales(gpu):
    """Scale bytes at both ends of the range, and their product back inside the output's."""
    _say("mx extreme scales")
    rng = np.random.default_rng(6)
    n, m, b = 40, 128, 3
    wc, ws = O.quantize(rng.standard_normal((n, m)), "e2m1")
    xc, xs = O.quantize(rng.standard_normal((b, m)), "e2m1")
    for dw, dx in ((120, -118), (-124, 122), (-60, 62)):
        W2 = np.clip(ws.astype(int) + dw, 0, 254).astype(np.uint8)
        X2 = np.clip(xs.astype(int) + dx, 0, 254).astype(np.uint8)
        ref, mag = O.linear(O.values(xc, X2, "e2m1"), O.values(wc, W2, "e2m1"))
        L = dbf.Layer.mx(blocks_to_dev(wc, W2, m, "e2m1"), max_batch=b)
        try:
            y = L.forward(blocks_to_dev(xc, X2, m, "e2m1"), out_dtype=T("bf16"))
            check(y, ref, mag, m, "bf16", True)
        finally:
            L.close()


@pytest.mark.parametrize("b", [1, 9, 33, 200])
def test_call_forms_agree(gpu, b):
    """dbf_linear_forward(_ex), grouped and allocation-free forwards: the bits of the layer's own forward."""
    torch = _torch()
    _say(f"mx call forms b={b}")
    rng = np.random.default_rng(b)
    m = 520
    layers = [dbf.Layer.mx(weight(rng, n, m)[0], max_batch=b, act=act)
              for n, act in ((256, "e4m3"), (96, "e4m3"), (33, "e2m1"), (300, "e2m1"))]
    R = inputs.random_layer("mx mixed", 64, m, 128, 0, 0.05, 0.05, 0.05, (b,))
    signs = dbf.Layer(R.A, R.B, R.a, R.mid, R.b, max_batch=b)
    try:
        xd, _ = to_dev(rows_of(rng, b, m), "f16")
        own = [L(xd) for L in layers]
        for ys in (dbf.forward_group(layers, xd), dbf.forward_group(layers[:1], xd)):
            for y, o in zip(ys, own):
                assert same_bits(y, o)
        mixed = dbf.forward_group([layers[0], signs, layers[2]], xd)
        assert same_bits(mixed[0], own[0]) and same_bits(mixed[1], signs(xd)) and same_bits(mixed[2], own[2])
        st = torch.cuda.current_stream().cuda_stream
        for L, o in zip(layers, own):
            y = torch.empty_like(o)
            dbf.dbf_linear_forward(L.handle, xd.data_ptr(), y.data_ptr(), b, st)
            assert same_bits(y, o)
            # (the first call on a device resolves the scratch array's address there)
            dbf.dbf_linear_forward_noalloc(L.handle, xd.data_ptr(), y.data_ptr(), b, st)
            y.zero_()
            torch.cuda.synchronize()
            free0 = torch.cuda.mem_get_info()[0]
            dbf.dbf_linear_forward_noalloc(L.handle, xd.data_ptr(), y.data_ptr(), b, st)
            torch.cuda.synchronize()
            assert torch.cuda.mem_get_info()[0] == free0
            assert same_bits(y, o)
            assert same_bits(L.forward(xd, path=dbf.DBF_PATH_PREFILL), o)
        dbf.dbf_timing_enable(layers[0].handle, True)
        assert same_bits(layers[0](xd), own[0])
        names = dbf.dbf_timing_read(layers[0].handle)
        assert names and all(v["launches"] >= 1 for v in names.values())
    finally:
        for L in layers + [signs]:
            L.close()


@pytest.mark.parametrize("b", [1, 5, 40, 300])
def test_group_of_blocks_and_bf16(gpu, b):
    """Layers that share blocks of either format, or bf16 rows: the bits of each layer's own forward."""
    torch = _torch()
    _say(f"mx group b={b}")
    rng = np.random.default_rng(b)
    m = 1000
    layers = [dbf.Layer.mx(weight(rng, n, m)[0], max_batch=b, act=act)
              for n, act in ((256, "e4m3"), (33, "e2m1"), (300, "e4m3"))]
    try:
        xd, _ = to_dev(rows_of(rng, b, m), "bf16")
        for x in (xd, dbf.mx_quantize(xd, "e4m3"), dbf.mx_quantize(xd, "e2m1")):
            for t in (torch.float16, torch.bfloat16):
                own = [L.forward(x, out_dtype=t) for L in layers]
                for y, o in zip(dbf.forward_group(layers, x, out_dtype=t), own):
                    assert y.dtype == t and same_bits(y, o)
                outs = [torch.empty_like(o) for o in own]
                assert dbf.forward_group(layers, x, outs=outs)[0] is outs[0]
                for y, o in zip(outs, own):
                    assert same_bits(y, o)
        with pytest.raises(ValueError):
            dbf.forward_group(layers, xd, outs=[torch.empty_like(o) for o in own[:2]])
        with pytest.raises(ValueError):
            dbf.forward_group(layers, xd[:, :512].contiguous())
        with pytest.raises(ValueError):
            dbf.forward_group(layers, xd, out_dtype=torch.float32)
        with pytest.raises(dbf.DbfError):
            dbf.forward_group(layers, torch.cat([xd, xd]))  # above max_batch
    finally:
        for L in layers:
            L.close()


@pytest.mark.parametrize("b", [1, 3, 16, 70])
@pytest.mark.parametrize("name", ["f16", "bf16"])
def test_norm_in_front_of_a_group(gpu, b, name):
    """Norm and the layers behind it: blocks where all take e4m3, 16 bits otherwise, sign layers among them."""
    torch = _torch()
    _say(f"norm and group b={b} {name}")
    rng = np.random.default_rng(b)
    m = 256
    up, gate = (dbf.Layer.mx(weight(rng, 400, m)[0], max_batch=b) for _ in range(2))
    low = dbf.Layer.mx(weight(rng, 96, m)[0], max_batch=b, act="e2m1")
    R = inputs.random_layer("norm group", 64, m, 128, 0, 0.05, 0.05, 0.05, (b,))
    signs = dbf.Layer(R.A, R.B, R.a, R.mid, R.b, max_batch=b)
    try:
        x, _ = to_dev(rows_of(rng, b, m), name)
        r, _ = to_dev(rows_of(rng, b, m), name)
        w, _ = to_dev(1 + 0.1 * rng.standard_normal(m), name)
        q = dbf.rms_norm(x, w, residual=r, eps=1e-5, mx=True)
        ys, norm = dbf.norm_forward_group([up, gate], x, w, residual=r, eps=1e-5)
        assert isinstance(norm.y, dbf.MxTensor) and torch.equal(norm.y.codes, q.y.codes) and same_bits(norm.h, q.h)
        for y, L in zip(ys, (up, gate)):
            assert y.dtype == x.dtype and same_bits(y, L.forward(q.y, out_dtype=x.dtype))
        plain = dbf.rms_norm(x, w, residual=r, eps=1e-5)
        ys, norm = dbf.norm_forward_group([up, low], x, w, residual=r, eps=1e-5)
        assert same_bits(norm.y, plain.y)
        for y, L in zip(ys, (up, low)):
            assert same_bits(y, L(plain.y))
        if name == "f16":
            ys, norm = dbf.norm_forward_group([signs, up], x, w, residual=r, eps=1e-5)
            for y, L in zip(ys, (signs, up)):
                assert same_bits(y, L(plain.y))
        else:
            with pytest.raises(ValueError):
                dbf.norm_forward_group([signs, up], x, w, residual=r)
    finally:
        for L in (up, gate, low, signs):
            L.close()


@pytest.mark.parametrize("b,m", [(16, 9216), (16, 8192), (13, 4100), (4, 16512)])
def test_call_forms_agree_at_wide_inputs(gpu, b, m):
    """Few rows on either side of what fits LDS, of what the product quantises itself, and of the widest input."""
    torch = _torch()
    _say(f"mx call forms b={b} m={m}")
    rng = np.random.default_rng(b + m)
    layers = [dbf.Layer.mx(weight(rng, n, m)[0], max_batch=b, act=act)
              for n, act in ((70, "e4m3"), (33, "e2m1"), (70, "e4m3"))]
    try:
        xd, _ = to_dev(rows_of(rng, b, m), "f16")
        own = [L(xd) for L in layers]
        for L, o in zip(layers, own):
            assert same_bits(L(dbf.mx_quantize(xd, L.act)), o)
            y = torch.empty_like(o)
            dbf.dbf_linear_forward_noalloc(L.handle, xd.data_ptr(), y.data_ptr(), b,
                                           torch.cuda.current_stream().cuda_stream)
            assert same_bits(y, o)
        # the same handle twice in a group too
        for y, o in zip(dbf.forward_group(layers + layers[:1], xd), own + own[:1]):
            assert same_bits(y, o)
    finally:
        for L in layers:
            L.close()


def test_handle_refusals(gpu):
    torch = _torch()
    _say("mx handle refusals")
    rng = np.random.default_rng(1)
    W, _ = weight(rng, 40, 64)
    L = dbf.Layer.mx(W, max_batch=4)
    R = inputs.random_layer("mx refuse", 32, 64, 64, 0, 0.05, 0.05, 0.05, (4,))
    S = dbf.Layer(R.A, R.B, R.a, R.mid, R.b, max_batch=4)
    lib = dbf.lib()
    E, U = dbf.DBF_ERR_INVALID_ARG, dbf.DBF_ERR_UNSUPPORTED
    try:
        x = torch.zeros(4, 64, dtype=torch.float16, device="cuda")
        y = torch.empty(4, 40, dtype=torch.float16, device="cuda")
        s = torch.zeros(4, 4, dtype=torch.uint8, device="cuda")
        X, Y, SC = x.data_ptr(), y.data_ptr(), s.data_ptr()
        f = lib.dbf_mx_forward
        assert f(L.handle, X, 0, None, Y, 0, 5, None) == E          # batch above max_batch
        assert f(L.handle, X, 0, None, Y, 0, -1, None) == E
        assert f(L.handle, X, 0, None, Y, 0, 0, None) == dbf.DBF_OK
        assert f(L.handle, X, 2, None, Y, 0, 4, None) == E          # fp32 rows
        assert f(L.handle, X, 0, None, Y, 2, 4, None) == E
        assert f(L.handle, X, 0, SC, Y, 0, 4, None) == E            # scales with 16-bit rows
        assert f(L.handle, X, 3, None, Y, 0, 4, None) == E          # blocks without scales
        assert f(L.handle, X + 2, 0, None, Y, 0, 4, None) == E
        assert f(L.handle, X, 0, None, None, 0, 4, None) == E
        assert f(S.handle, X, 0, None, Y, 0, 4, None) == U          # not a block layer
        assert lib.dbf_mx_backward_data(S.handle, Y, X, 0, 4, None) == U
        assert lib.dbf_mx_backward_data(L.handle, Y, X, 2, 4, None) == E
        assert lib.dbf_mx_backward_data(L.handle, Y, X, 0, 5, None) == E
        assert lib.dbf_linear_forward_ex(L.handle, X, Y, 4, dbf.DBF_PATH_DECODE_EXACT, None) == U
        assert lib.dbf_linear_forward_ex(L.handle, X, Y, 4, dbf.DBF_PATH_DECODE_TABLE, None) == U
        assert lib.dbf_linear_backward(L.handle, X, Y, X, None, None, None, 4, None) == U
        with pytest.raises(ValueError):
            L(x.float())
        with pytest.raises(ValueError):
            L(x[:, :32])
        with pytest.raises(ValueError):
            L.forward(x, out_dtype=torch.float32)
        with pytest.raises(ValueError):
            L.forward(x, out=y[:2])
        with pytest.raises(ValueError):
            S.forward(x, out_dtype=torch.bfloat16)
        with pytest.raises(ValueError):
            L.backward_data(x)
        with pytest.raises(dbf.DbfError):
            L.forward(x, path=dbf.DBF_PATH_DECODE_EXACT)
        info = L.info()
        assert (info["n"], info["m"], info["k"], info["n_pad"], info["m_pad"]) == (40, 64, 0, 64, 128)
        assert info["packed_bytes"] == 64 * 64
    finally:
        L.close()
        S.close()


def test_pack_out_of_memory_leaks_nothing(gpu, monkeypatch):
    torch = _torch()
    _say("mx pack allocation failures")
    W, _ = weight(np.random.default_rng(2), 4096, 4096)
    L = dbf.Layer.mx(W, max_batch=64)
    L.close()
    torch.cuda.synchronize()
    free0 = torch.cuda.mem_get_info()[0]
    failed = 0
    for i in range(1, 12):
        monkeypatch.setenv("DBF_TEST_FAIL_ALLOC", str(i))
        try:
            L = dbf.Layer.mx(W, max_batch=64)
            L.close()
            break
        except dbf.DbfError as e:
            assert e.status == dbf.DBF_ERR_OOM
            failed += 1
    assert failed >= 3
    assert torch.cuda.mem_get_info()[0] == free0


# ---------------------------------------------------------------- the gradient

@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("b,n,m", [(1, 1, 1), (1, 64, 32), (3, 33, 31), (16, 100, 129), (17, 256, 640), (40, 1000, 130),
                                   (64, 77, 512), (129, 320, 300), (257, 513, 520)])
def test_backward_data(gpu, b, n, m, name):
    """f16 / bf16 products are exact in fp32 (11 and 2 bits); sums of n of them in fp32."""
    _say(f"mx backward b={b} n={n} m={m} {name}")
    rng = np.random.default_rng(b + 5 * n + m)
    W, wv = weight(rng, n, m)
    dyd, dyv = to_dev(rows_of(rng, b, n, 0.1), name)
    ref, mag = O.backward_data(dyv, wv)
    L = dbf.Layer.mx(W, max_batch=b)
    try:
        dx = L.backward_data(dyd)
        assert dx.dtype == T(name) and tuple(dx.shape) == (b, m)
        # a matrix-core step adds 16 products at most at once: n / 8 additions in a row at most
        acc = (n / 8 + 4) * 2.0 ** -24
        tol = half_step(name) * (np.abs(ref) + acc * mag) + acc * mag + tiny(name)
        d = np.abs(dx.double().cpu().numpy() - ref)
        assert np.all(d <= tol), float((d / tol).max())
        if name == "f16":
            st = _torch().cuda.current_stream().cuda_stream
            dx2 = _torch().empty_like(dx)
            dbf.dbf_linear_backward_data(L.handle, dyd.data_ptr(), dx2.data_ptr(), b, st)
            assert same_bits(dx, dx2)
    finally:
        L.close()


@pytest.mark.parametrize("b,n,m,name", [(1900, 1032, 8100, "bf16"), (1900, 1030, 8100, "f16"), (700, 2008, 2050, "f16"),
                                        (700, 2001, 2050, "bf16"), (300, 4104, 1000, "bf16"), (33, 4099, 900, "f16"),
                                        (1900, 40, 8100, "f16"), (1900, 100, 8100, "bf16"), (1900, 1024, 8100, "bf16"),
                                        (1900, 64, 8100, "f16"), (1900, 192, 8100, "bf16"), (700, 2048, 2050, "f16"),
                                        (300, 4096, 1000, "bf16"), (33, 4096, 900, "f16"), (5, 64, 100, "bf16")])
def test_backward_large(gpu, b, n, m, name):
    """Every tile, whole and in K parts, fewer steps than the pipeline holds, rows that are not 16-byte aligned."""
    _say(f"mx backward large b={b} n={n} m={m} {name}")
    rng = np.random.default_rng(b + n + m)
    W, wv = weight(rng, n, m)
    dyd, dyv = to_dev(rows_of(rng, b, n, 0.1), name)
    ref, mag = _device_products(dyv, wv.T)
    L = dbf.Layer.mx(W, max_batch=b)
    try:
        dx = L.backward_data(dyd)
        acc = (n / 8 + 4) * 2.0 ** -24
        tol = half_step(name) * (np.abs(ref) + acc * mag) + acc * mag + tiny(name)
        d = np.abs(dx.double().cpu().numpy() - ref)
        assert np.all(d <= tol), float((d / tol).max())
        for _ in range(3):
            assert same_bits(L.backward_data(dyd), dx)
    finally:
        L.close()


def test_backward_non_finite_rows(gpu):
    """An infinity or a NaN of dy stays in its row, also beside the end of the rows."""
    _say("mx backward non-finite")
    torch = _torch()
    rng = np.random.default_rng(9)
    n, m, b = 72, 96, 70
    W, _ = weight(rng, n, m)
    dy, _ = to_dev(rng.standard_normal((b, n)), "bf16")
    L = dbf.Layer.mx(W, max_batch=b)
    try:
        clean = L.backward_data(dy)
        dy[3, 0] = float("nan")
        dy[40, 70] = float("inf")
        dx = L.backward_data(dy)
        keep = torch.ones(b, dtype=torch.bool)
        keep[[3, 40]] = False
        assert same_bits(dx[keep.cuda()], clean[keep.cuda()])
        assert bool(torch.isnan(dx[3]).all()) and not bool(torch.isfinite(dx[40]).any())
    finally:
        L.close()


def test_backward_scale_range(gpu):
    """Rows of the weight whose scales differ by 2^24 inside a block column: the small ones still count in f16
    (alone in their column), and a NaN block makes its columns NaN."""
    _say("mx backward scales")
    rng = np.random.default_rng(8)
    n, m, b = 96, 64, 5
    wc, ws = O.quantize(rng.standard_normal((n, m)), "e2m1")
    ws = ws.astype(int)
    ws[:48] -= 24
    ws = ws.astype(np.uint8)
    wc[48:, 7] = 0  # column 7: only the small rows
    dyd, dyv = to_dev(rng.standard_normal((b, n)), "bf16")
    wv = O.values(wc, ws, "e2m1")
    ref, mag = O.backward_data(dyv, wv)
    for name in ("bf16", "f16"):
        dyd, dyv = to_dev(dyv, name)
        L = dbf.Layer.mx(blocks_to_dev(wc, ws, m, "e2m1"), max_batch=b)
        try:
            dx = L.backward_data(dyd).double().cpu().numpy()
        finally:
            L.close()
        acc = (n / 8 + 4) * 2.0 ** -24
        assert np.all(np.abs(dx - ref) <= half_step(name) * (np.abs(ref) + acc * mag) + acc * mag + tiny(name))
    ws[50, 1] = 255
    L = dbf.Layer.mx(blocks_to_dev(wc, ws, m, "e2m1"), max_batch=b)
    try:
        dx = L.backward_data(dyd).cpu().numpy()
        assert np.isnan(dx[:, 32:]).all() and np.isfinite(dx[:, :32]).all()
    finally:
        L.close()


@pytest.mark.parametrize("name", ["bf16", "f16"])
def test_backward_smallest_exact_scales(gpu, name):
    """Scales of 2^-28 of the block column's largest: every code still exact (2^-16 and up in 16 bits)."""
    _say(f"mx backward smallest scales {name}")
    rng = np.random.default_rng(9)
    n, m, b = 128, 64, 7
    wc = rng.integers(0, 16, size=(n, m)).astype(np.uint8)
    ws = np.full((n, m // 32), 127 - 28, dtype=np.uint8)
    ws[64:] = 127
    wc[64:] = 0          # (the large rows are zeros: what is left is the small ones alone)
    wc[64:, ::32] = 1
    dyd, dyv = to_dev(rng.integers(-64, 65, size=(b, n)) * 2.0 ** 8, name)
    wv = O.values(wc, ws, "e2m1")
    ref, _ = O.backward_data(dyv, wv)
    L = dbf.Layer.mx(blocks_to_dev(wc, ws, m, "e2m1"), max_batch=b)
    try:
        dx = L.backward_data(dyd).double().cpu().numpy()
    finally:
        L.close()
    cols = np.arange(m) % 32 != 0
    # whole numbers of 2^-21 below 2^24 of them: the fp32 sums are exact, one rounding is left
    assert np.all(np.abs(dx - ref)[:, cols] <= half_step(name) * np.abs(ref)[:, cols] + tiny(name))


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("rows", [1, 7, 130])
def test_block_of_a_decoder(gpu, rows):
    """norm -> grouped gate and up -> norm -> down, with each layer's input gradient: run as a model runs them,
    eager, on another stream, and captured and replayed."""
    torch = _torch()
    _say(f"mx decoder block rows={rows}")
    rng = np.random.default_rng(rows)
    d, f = 384, 1000
    gate, gv = weight(rng, f, d)
    up, uv = weight(rng, f, d)
    down, dv = weight(rng, d, f)
    Lg, Lu, Ld = (dbf.Layer.mx(w, max_batch=rows) for w in (gate, up, down))
    x, xv = to_dev(rows_of(rng, rows, d), "f16")
    r, rv = to_dev(rows_of(rng, rows, d), "f16")
    w, wv = to_dev(1 + 0.1 * rng.standard_normal(d), "f16")

    def step():
        a = dbf.rms_norm(x, w, residual=r, eps=1e-5, mx=True)
        g, u = Lg.forward(a.y), Lu.forward(a.y)
        z = g * u
        y = Ld(z)
        dz = Ld.backward_data(y)
        dxn, dwn = dbf.rms_norm_backward(Lg.backward_data(dz), a.h, w, a.rstd, dh=y)
        return a.h, g, u, z, y, dz, dxn, dwn

    try:
        eager = step()
        h = (xv + rv).astype(np.float16).astype(np.float64)
        assert np.array_equal(eager[0].double().cpu().numpy(), h)
        # each layer's product of what it was given
        a = dbf.rms_norm(x, w, residual=r, eps=1e-5, mx=True)
        ac, as_ = O.unpad_rows(a.y.codes.cpu().numpy(), a.y.scales.cpu().numpy(), d, "e4m3")
        for got, vals in ((eager[1], gv), (eager[2], uv)):
            ref, mag = O.linear(O.values(ac, as_, "e4m3"), vals)
            check(got, ref, mag, d, "f16", False)
        zc, zs = O.quantize(eager[3].double().cpu().numpy(), "e4m3")
        ref, mag = O.linear(O.values(zc, zs, "e4m3"), dv)
        check(eager[4], ref, mag, f, "f16", False)
        # another stream
        s2 = torch.cuda.Stream()
        s2.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s2):
            other = step()
        s2.synchronize()
        for p, q in zip(eager, other):
            assert same_bits(p, q)
        # captured: three replays, with eager work between
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()
        for _ in range(3):
            for t in held:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            for p, q in zip(eager, held):
                assert same_bits(p, q)
            again = step()
            for p, q in zip(eager, again):
                assert same_bits(p, q)
    finally:
        for L in (Lg, Lu, Ld):
            L.close()
