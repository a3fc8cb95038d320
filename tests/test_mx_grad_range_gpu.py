"""GPU: input gradients of a 4-bit layer over the whole range of the types.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as O
from tests.test_mx_gpu import blocks_to_dev, half_step, rows_of, tiny, to_dev, weight

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("b,n,m", [(3, 64, 96), (40, 100, 129), (130, 72, 300), (300, 4096, 200)])
@pytest.mark.parametrize("power", [-100, 60, 110, 114])
def test_rows_of_any_magnitude(gpu, b, n, m, power):
    """bf16 gradients up to a sum of magnitudes that, times the largest code, fits fp32; the tolerance is that of
    ordinary ones (products exact, at most n / 8 additions of fp32 in a row)."""
    _say(f"mx backward magnitude b={b} n={n} m={m} 2^{power}")
    rng = np.random.default_rng(b + n + m)
    W, wv = weight(rng, n, m)
    dyd, dyv = to_dev(np.clip(rows_of(rng, b, n, 0.1), -4, 4) * 2.0 ** power, "bf16")
    assert 6 * np.abs(dyv).sum(axis=1).max() < 2.0 ** 128
    ref, mag = O.backward_data(dyv, wv)
    L = dbf.Layer.mx(W, max_batch=b)
    try:
        dx = L.backward_data(dyd).double().cpu().numpy()
    finally:
        L.close()
    acc = (n / 8 + 4) * 2.0 ** -24
    tol = half_step("bf16") * (np.abs(ref) + acc * mag) + acc * mag + tiny("bf16")
    d = np.abs(dx - ref)
    assert np.all(d <= tol), float((d / tol).max())


@pytest.mark.parametrize("b,n,m", [(7, 192, 96), (130, 1030, 300)])
@pytest.mark.parametrize("name,low", [("f16", 36), ("bf16", 125)])
def test_smallest_exact_scales(gpu, name, low, b, n, m):
    """Scales of 2^-36 (f16) and 2^-125 (bf16) of the block column's largest: every code enters exactly (0.5 is then
    f16's smallest number and bf16's smallest normal one), the sums of whole numbers are exact in fp32, and one
    rounding is left."""
    _say(f"mx backward smallest scales {name} 2^-{low} b={b} n={n} m={m}")
    rng = np.random.default_rng(low)
    wc = rng.integers(0, 16, size=(n, m)).astype(np.uint8)
    ws = np.full((n, -(-m // 32)), 127, dtype=np.uint8)
    ws[-64:] = 127 + low
    wc[-64:] = 0  # the large rows only set the common exponent
    dyd, dyv = to_dev(rng.integers(-4, 5, size=(b, n)).astype(np.float64), name)
    ref, mag = O.backward_data(dyv, O.values(wc, ws, "e2m1"))
    assert (2 * mag).max() < 2 ** 24 and np.abs(ref).max() < 65504
    L = dbf.Layer.mx(blocks_to_dev(wc, ws, m, "e2m1"), max_batch=b)
    try:
        dx = L.backward_data(dyd).double().cpu().numpy()
    finally:
        L.close()
    assert np.all(np.abs(dx - ref) <= half_step(name) * np.abs(ref))
