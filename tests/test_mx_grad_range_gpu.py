"""GPU: input gradients of a 4-bit layer over the whole range of the types.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as O
from tests.test_mx_gpu import half_step, rows_of, tiny, to_dev, weight

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
