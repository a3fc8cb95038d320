"""GPU: the norm over rows of any magnitude: their squares are formed in 64 bits.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from tests.test_mx_gpu import same_bits, to_dev

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


# powers of two that keep whole numbers up to 8 exact in the type, and the row's 1 / rms a normal fp32 number
POWERS = {"bf16": (-127, -120, -80, -70, -60, 60, 62, 64, 100, 121), "f16": (-24, -14, 9, 12)}


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
        # one rounding to fp32 (and 2^-40 for the arithmetic in 64 bits)
        assert np.all(np.abs(got - rstd) <= (2.0 ** -24 + 2.0 ** -40) * rstd), k


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
