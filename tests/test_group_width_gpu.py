"""GPU: a grouped forward refuses rows of another width than its layers', before it launches anything."""

import pytest

import dbf_linear_fwd_amd as dbf
from tests import inputs
from tests.test_mx_gpu import weight

pytestmark = pytest.mark.gpu


def test_rows_of_another_width(gpu):
    import numpy as np
    import torch
    print("[case] group width", flush=True)
    R = inputs.random_layer("group width", 64, 128, 128, 0, 0.05, 0.05, 0.05, (2,))
    signs = dbf.Layer(R.A, R.B, R.a, R.mid, R.b, max_batch=2)
    rng = np.random.default_rng(0)
    up, low = (dbf.Layer.mx(weight(rng, 96, m)[0], max_batch=2) for m in (128, 64))
    try:
        x = torch.zeros((2, 128), dtype=torch.float16, device="cuda")
        for layers in ([signs], [signs, up], [up], [up, signs]):
            for w in (64, 120, 136):
                with pytest.raises(ValueError, match="width|columns"):
                    dbf.forward_group(layers, torch.zeros((2, w), dtype=torch.float16, device="cuda"))
            assert len(dbf.forward_group(layers, x)) == len(layers)
        with pytest.raises(ValueError):
            dbf.forward_group([signs, low], x)
        with pytest.raises(dbf.DbfError):
            dbf.forward_group([up, low], x)
    finally:
        for L in (signs, up, low):
            L.close()
