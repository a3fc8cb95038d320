"""GPU: grouped forwards of 4-bit layers into outputs of either 16-bit type.

Every case prints its name before it touches the GPU.
"""

import sys

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from tests import inputs
from tests.test_mx_gpu import T, rows_of, same_bits, to_dev, weight

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


@pytest.mark.parametrize("b", [1, 20])
@pytest.mark.parametrize("rows,out", [("f16", "bf16"), ("bf16", "f16"), ("f16", "f16"), ("bf16", "bf16")])
def test_outputs_give_their_type(gpu, b, rows, out):
    """Without out_dtype the results take the outputs' type, as a single layer's do."""
    import torch
    _say(f"mx group outputs b={b} {rows} to {out}")
    rng = np.random.default_rng(b)
    m = 256
    layers = [dbf.Layer.mx(weight(rng, n, m)[0], max_batch=b, act=act)
              for n, act in ((96, "e4m3"), (33, "e2m1"), (64, "e4m3"))]
    try:
        x, _ = to_dev(rows_of(rng, b, m), rows)
        w, _ = to_dev(1 + 0.1 * rng.standard_normal(m), rows)
        new = lambda ls: [torch.empty((b, L.n), dtype=T(out), device="cuda") for L in ls]  # noqa: E731
        want = [L.forward(x, out=y) for L, y in zip(layers, new(layers))]
        outs = new(layers)
        assert all(a is b_ for a, b_ in zip(dbf.forward_group(layers, x, outs=outs), outs))
        for y, o in zip(outs, want):
            assert same_bits(y, o)
        # the norm in front: its rows in 16 bits (a layer takes e2m1), and in blocks (all take e4m3)
        for ls in (layers, [layers[0], layers[2]]):
            outs = new(ls)
            ys, norm = dbf.norm_forward_group(ls, x, w, outs=outs)
            assert isinstance(norm.y, dbf.MxTensor) == (len(ls) == 2)
            for y, o, L in zip(ys, outs, ls):
                assert y is o and same_bits(y, L.forward(norm.y, out_dtype=T(out)))
        # outputs of two types are refused
        outs = new(layers)
        outs[1] = outs[1].to(T("f16" if out == "bf16" else "bf16"))
        with pytest.raises(ValueError):
            dbf.forward_group(layers, x, outs=outs)
        with pytest.raises(ValueError):
            dbf.forward_group(layers, x, outs=new(layers), out_dtype=T("f16" if out == "bf16" else "bf16"))
    finally:
        for L in layers:
            L.close()


def test_sign_layers_take_float16(gpu):
    """A group with a sign layer: float16 rows into float16 outputs; anything else is refused, and in front of the
    norm, before it runs."""
    import torch
    _say("mx group outputs with a sign layer")
    rng = np.random.default_rng(0)
    m = 128
    R = inputs.random_layer("group outputs", 64, m, 128, 0, 0.05, 0.05, 0.05, (2,))
    signs = dbf.Layer(R.A, R.B, R.a, R.mid, R.b, max_batch=2)
    up = dbf.Layer.mx(weight(rng, 96, m)[0], max_batch=2)
    try:
        x, _ = to_dev(rows_of(rng, 2, m), "f16")
        outs = [torch.empty((2, L.n), dtype=torch.bfloat16, device="cuda") for L in (signs, up)]
        with pytest.raises(ValueError):
            dbf.forward_group([signs, up], x, outs=outs)
        with pytest.raises(ValueError):
            dbf.norm_forward_group([signs, up], x.bfloat16())
        ys = dbf.forward_group([signs, up], x)
        assert same_bits(ys[0], signs(x)) and same_bits(ys[1], up(x))
    finally:
        signs.close()
        up.close()
