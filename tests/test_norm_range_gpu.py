"""GPU: the norm over rows of any magnitude, and its block codes next to a rounding border: statistics in 64 bits.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as O
from tests.test_mx_gpu import same_bits, to_dev

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


# powers of two that keep whole numbers up to 8 exact in the type (the smallest: 1 / rms is above fp32's range)
POWERS = {"bf16": (-133, -130, -127, -120, -80, -70, -60, 60, 62, 64, 100, 121), "f16": (-24, -14, 9, 12)}


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("cols", [8, 40, 1001, 2048, 5000, 16392])
def test_rows_of_any_magnitude(gpu, cols, name):
    """With eps = 0 a row times a power of two has the row's result: every step but the last scales exactly."""
    import torch
    _say(f"norm magnitudes {cols} {name}")
    rng = np.random.default_rng(cols)
    x = rng.integers(-7, 8, size=(3, cols)).astype(np.float64)
    x[:, 0] = 8.0
    w, _ = to_dev(1 + 0.2 * rng.standard_normal(cols), "f32")
    xd, _ = to_dev(x, name)
    want, want_q = dbf.rms_norm(xd, w, eps=0.0), dbf.rms_norm(xd, w, eps=0.0, mx=True)
    assert bool(torch.isfinite(want.y).all()) and bool((want.y != 0).any())
    for k in POWERS[name]:
        v, held = to_dev(x * 2.0 ** k, name)
        assert np.array_equal(held, x * 2.0 ** k), k
        out, q = dbf.rms_norm(v, w, eps=0.0), dbf.rms_norm(v, w, eps=0.0, mx=True)
        assert same_bits(out.y, want.y), k
        assert torch.equal(q.y.codes, want_q.y.codes) and torch.equal(q.y.scales, want_q.y.scales), k
        rstd = 1 / np.sqrt((held * held).mean(axis=1))
        got = out.rstd.double().cpu().numpy()
        if rstd.max() < 2.0 ** 128:
            # one rounding to fp32 (and 2^-40 for the arithmetic in 64 bits)
            assert np.all(np.abs(got - rstd) <= (2.0 ** -24 + 2.0 ** -40) * rstd), k
        else:
            assert np.isinf(got[rstd >= 2.0 ** 128]).all(), k


def test_rows_of_mixed_magnitude(gpu):
    """Values whose squares vanish or overflow in 32 bits next to each other in a row."""
    _say("norm mixed magnitudes")
    rng = np.random.default_rng(1)
    for cols in (40, 3000):
        x = rng.standard_normal((4, cols)) * np.exp2(rng.integers(-110, 110, size=(4, cols)))
        xd, xv = to_dev(x, "bf16")
        y = dbf.rms_norm(xd, None, eps=0.0).y.double().cpu().numpy()
        ref = xv / np.sqrt((xv * xv).mean(axis=1, keepdims=True))
        # half a step and the fp32 rounding before it, among subnormal values half of their steps
        assert np.all(np.abs(y - ref) <= (2.0 ** -8 + 2.0 ** -23) * np.abs(ref) + 2.0 ** -134 + 2.0 ** -149)


def codes_of_nearby(codes, ref):
    """How many codes no value within one fp32 rounding of ref has (2^-24 of it; 2^-40 for the arithmetic in 64
    bits).  ref: the exact values over their block's scale."""
    rel = 2.0 ** -24 + 2.0 ** -40
    got = np.abs(O.code_values("e4m3")[codes])
    lo = O.code_values("e4m3")[O.nearest_code(np.abs(ref) * (1 - rel), "e4m3")]
    hi = O.code_values("e4m3")[O.nearest_code(np.abs(ref) * (1 + rel), "e4m3")]
    return int(((got < lo) | (got > hi)).sum())


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("cols", [96, 1000, 4096])
def test_block_codes_next_to_ties(gpu, cols, name):
    """Values within a few 2^-24 of the middle between two codes.  The value that is quantised is the exact one
    rounded to fp32 once (2^-24 of it; the arithmetic in 64 bits adds less than 2^-40): a code is right if some
    value that near to the exact one has it."""
    import torch
    _say(f"norm ties {cols} {name}")
    rng = np.random.default_rng(cols)
    rows = 4
    h = np.exp2(rng.uniform(-2, 2, size=cols)) * rng.choice([-1.0, 1.0], size=cols)
    hd, hv = to_dev(np.tile(h, (rows, 1)), name)
    rstd = 1 / np.sqrt((hv[0] * hv[0]).mean() + float(np.float32(1e-5)))
    xh = hv[0] * rstd
    table = O.code_values("e4m3")[:127].astype(np.float64)
    # the first column of a block sets the scale to 1 (a largest value of 256 to 448), the others lie next to a tie
    i = rng.integers(8, 118, size=cols)
    target = (table[i] + table[i + 1]) / 2 * (1 + rng.uniform(-4, 4, size=cols) * 2.0 ** -24)
    target[::32] = 300.0
    wd, wv = to_dev(target / np.abs(xh), "f32")
    assert wv.max() < 2.0 ** 30
    ref = hv * rstd * wv
    q = dbf.rms_norm(hd, wd, eps=1e-5, mx=True)
    codes, s = O.unpad_rows(q.y.codes.cpu().numpy(), q.y.scales.cpu().numpy(), cols, "e4m3")
    assert np.all(s == 127)
    assert codes_of_nearby(codes, ref) == 0
    assert torch.equal(q.y.codes[0], q.y.codes[rows - 1])


@pytest.mark.parametrize("name", ["f16", "bf16"])
@pytest.mark.parametrize("rows,cols", [(1024, 4096), (3000, 1000), (500, 8200)])
def test_block_codes_of_many(gpu, rows, cols, name):
    """Weights of the rows' own type or none: some millions of values, a few of them next to a border by chance."""
    _say(f"norm codes {rows}x{cols} {name}")
    rng = np.random.default_rng(rows)
    hd, hv = to_dev(rng.standard_normal((rows, cols)), name)
    for wd, wv in (to_dev(1 + 0.2 * rng.standard_normal(cols), name), (None, 1.0)):
        ref = hv * (1 / np.sqrt((hv * hv).mean(axis=1) + float(np.float32(1e-5))))[:, None] * wv
        q = dbf.rms_norm(hd, wd, eps=1e-5, mx=True)
        codes, s = O.unpad_rows(q.y.codes.cpu().numpy(), q.y.scales.cpu().numpy(), cols, "e4m3")
        inv = np.exp2(127.0 - np.repeat(s.astype(np.float64), 32, axis=1)[:, :cols])
        assert codes_of_nearby(codes, ref * inv) == 0
