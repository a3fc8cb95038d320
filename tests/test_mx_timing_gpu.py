"""GPU: kernel timing of layers with a 4-bit block weight: one entry for every kernel of a call, each with its own time.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from tests.test_mx_gpu import rows_of, to_dev, weight

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def _timed(L, call, times):
    """dbf_timing_read of `times` calls, the first call on the handle aside."""
    call()
    dbf.dbf_timing_enable(L.handle, True)
    try:
        dbf.dbf_timing_read(L.handle)
        for _ in range(times):
            call()
        return dbf.dbf_timing_read(L.handle)
    finally:
        dbf.dbf_timing_enable(L.handle, False)


@pytest.mark.parametrize("b,n,m,kernels", [
    (1, 64, 512, ["mx_decode"]),                                       # one launch
    (40, 4096, 256, ["mx_quantize", "mx_product"]),                    # K whole: two steps of 128 columns
    (16, 256, 14336, ["mx_quantize", "mx_product", "mx_product_join"]),  # K in parts
])
def test_forward_kernels(gpu, b, n, m, kernels):
    _say(f"mx timing forward b={b} n={n} m={m}")
    rng = np.random.default_rng(b + n + m)
    L = dbf.Layer.mx(weight(rng, n, m)[0], max_batch=b)
    try:
        x, _ = to_dev(rows_of(rng, b, m), "f16")
        got = _timed(L, lambda: L(x), 3)
        assert sorted(got) == sorted(kernels) and all(v["launches"] == 3 for v in got.values())
    finally:
        L.close()


@pytest.mark.parametrize("b,n,m,kernels", [(40, 128, 256, ["mx_backward"]),
                                           (300, 4096, 1000, ["mx_backward", "mx_backward_join"])])
def test_backward_kernels(gpu, b, n, m, kernels):
    _say(f"mx timing backward b={b} n={n} m={m}")
    rng = np.random.default_rng(b + n + m)
    L = dbf.Layer.mx(weight(rng, n, m)[0], max_batch=b)
    try:
        dy, _ = to_dev(rows_of(rng, b, n, 0.1), "bf16")
        got = _timed(L, lambda: L.backward_data(dy), 3)
        assert sorted(got) == sorted(kernels) and all(v["launches"] == 3 for v in got.values())
    finally:
        L.close()


def test_times_add_up(gpu):
    """A call of a hundred microseconds and more: its kernels' times are most of the time between two events around
    calls that follow each other (all but what lies between kernels, a few microseconds)."""
    import torch
    _say("mx timing sums")
    b, n, m = 512, 14336, 4096
    g = torch.Generator(device="cuda").manual_seed(1)
    w = 0.02 * torch.randn((n, m), generator=g, device="cuda")
    L = dbf.Layer.mx(dbf.mx_quantize(w, "e2m1"), max_batch=b)
    try:
        dy = torch.randn((b, n), generator=g, device="cuda").bfloat16()
        out = torch.empty((b, m), dtype=torch.bfloat16, device="cuda")
        call = lambda: L.backward_data(dy, out=out)  # noqa: E731
        for _ in range(5):
            call()
        start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(20):
            call()
        stop.record()
        stop.synchronize()
        got = _timed(L, call, 20)
        assert sorted(got) == ["mx_backward", "mx_backward_join"]
        total = sum(v["total_ms"] for v in got.values())
        assert total >= 0.5 * start.elapsed_time(stop), (got, start.elapsed_time(stop))
    finally:
        L.close()
