"""Argument checks of the block-format and norm entry points, on the host
(no GPU is needed: every call below is refused, or returns, before any HIP
call)."""

import ctypes

import pytest

import dbf_linear_fwd_amd as dbf

E = dbf.DBF_ERR_INVALID_ARG
P = ctypes.c_void_p(4096)      # aligned, never dereferenced
ODD = ctypes.c_void_p(4098)
F16, BF16, F32, E4M3, E2M1 = (dbf.DBF_TYPE_F16, dbf.DBF_TYPE_BF16, dbf.DBF_TYPE_F32, dbf.DBF_TYPE_E4M3,
                              dbf.DBF_TYPE_E2M1)


def test_row_bytes():
    L = dbf.lib()
    for cols in (1, 31, 32, 127, 128, 129, 4096, 14336):
        wide = -(-cols // 128) * 128
        assert L.dbf_mx_code_bytes(cols, E4M3) == wide
        assert L.dbf_mx_code_bytes(cols, E2M1) == wide // 2
        assert L.dbf_mx_scale_bytes(cols) == wide // 32
    assert L.dbf_mx_code_bytes(0, E4M3) == 0 and L.dbf_mx_code_bytes(64, F16) == 0
    assert L.dbf_mx_scale_bytes(-3) == 0 and L.dbf_mx_scale_bytes((1 << 30) + 1) == 0


def test_quantize_refusals():
    L = dbf.lib()
    for f in (lambda x, t, r, c, ft, q, s: L.dbf_mx_quantize(x, t, r, c, ft, q, s, None),
              lambda x, t, r, c, ft, q, s: L.dbf_mx_dequantize(q, s, ft, r, c, x, t, None)):
        assert f(P, F16, 0, 8, E4M3, P, P) == dbf.DBF_OK  # no rows: nothing to do
        assert f(None, F16, 4, 8, E4M3, P, P) == E
        assert f(P, F16, 4, 8, E4M3, None, P) == E
        assert f(P, F16, 4, 8, E4M3, P, None) == E
        assert f(ODD, F16, 4, 8, E4M3, P, P) == E
        assert f(P, F16, 4, 8, E4M3, ODD, P) == E
        assert f(P, F16, 4, 8, E4M3, P, ODD) == E
        assert f(P, F16, -1, 8, E4M3, P, P) == E
        assert f(P, F16, 4, 0, E4M3, P, P) == E
        assert f(P, E4M3, 4, 8, E4M3, P, P) == E
        assert f(P, 7, 4, 8, E4M3, P, P) == E
        assert f(P, F16, 4, 8, F16, P, P) == E
        assert f(P, F16, 1 << 30, 1 << 20, E4M3, P, P) == dbf.DBF_ERR_SHAPE
        assert f(P, F16, 1, (1 << 30) + 1, E4M3, P, P) == dbf.DBF_ERR_SHAPE


def test_pack_refusals():
    L = dbf.lib()
    h = ctypes.c_void_p()
    H = ctypes.byref(h)
    assert L.dbf_mx_pack(8, 8, P, P, E4M3, 4, None, None) == E
    assert L.dbf_mx_pack(8, 8, None, P, E4M3, 4, None, H) == E
    assert L.dbf_mx_pack(8, 8, P, None, E4M3, 4, None, H) == E
    assert L.dbf_mx_pack(8, 8, ODD, P, E4M3, 4, None, H) == E
    for n, m, b in ((0, 8, 4), (8, 0, 4), (8, 8, 0), (-1, 8, 4)):
        assert L.dbf_mx_pack(n, m, P, P, E4M3, b, None, H) == E
    assert L.dbf_mx_pack(8, 8, P, P, F16, 4, None, H) == E
    assert L.dbf_mx_pack((1 << 30) + 1, 8, P, P, E4M3, 4, None, H) == dbf.DBF_ERR_SHAPE
    assert L.dbf_mx_pack(1 << 20, 1 << 20, P, P, E4M3, 4, None, H) == dbf.DBF_ERR_SHAPE
    assert L.dbf_mx_pack(8, 1 << 20, P, P, E4M3, 1 << 20, None, H) == dbf.DBF_ERR_SHAPE
    assert h.value is None


def test_forward_and_backward_refuse_a_null_handle():
    L = dbf.lib()
    assert L.dbf_mx_forward(None, P, F16, None, P, F16, 1, None) == E
    assert L.dbf_mx_backward_data(None, P, P, F16, 1, None) == E


def test_forward_group_refusals():
    L = dbf.lib()
    one = (ctypes.c_void_p * 9)()
    ys = (ctypes.c_void_p * 9)(*[4096] * 9)
    f = lambda hs, n, y, b=1: L.dbf_mx_forward_group(hs, n, P, F16, None, y, F16, b, None)  # noqa: E731
    assert f(None, 1, ys) == E and f(one, 1, None) == E
    assert f(one, 0, ys) == E and f(one, 9, ys) == E and f(one, 1, ys, -1) == E
    assert f(one, 2, ys) == E  # null handles


def test_binding_group_refusals():
    import torch

    class Other:
        act, n, m = None, 8, 64

    for layers in ([Other()], []):
        for t in (torch.float16, torch.bfloat16):
            with pytest.raises(ValueError):
                dbf.forward_group(layers, torch.zeros(1, 64, dtype=t))
    with pytest.raises(ValueError):
        dbf.forward_group([Other()], torch.zeros(1, 64, dtype=torch.float16), out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dbf.norm_forward_group([Other()], torch.zeros(1, 64, dtype=torch.float16))


def _norm(x=P, r=None, w=P, t=F16, wt=F16, rows=4, cols=8, eps=1e-6, h=None, y=P, yt=F16, ys=None, rstd=None):
    return dbf.lib().dbf_rms_norm(x, r, w, t, wt, rows, cols, eps, h, y, yt, ys, rstd, None)


def test_norm_refusals():
    assert _norm(rows=0) == dbf.DBF_OK
    assert _norm(x=None) == E
    assert _norm(y=None) == E
    assert _norm(rows=-1) == E
    assert _norm(cols=0) == E
    assert _norm(cols=32769) == dbf.DBF_ERR_SHAPE
    assert _norm(t=F32) == E
    assert _norm(wt=BF16) == E
    assert _norm(yt=BF16) == E
    assert _norm(yt=dbf.DBF_TYPE_E2M1, ys=P) == E
    assert _norm(yt=E4M3) == E                       # scales missing
    assert _norm(eps=-1.0) == E
    assert _norm(eps=float("nan")) == E
    assert _norm(h=P) == E                           # h without a residual
    for k in ("x", "r", "w", "y", "rstd"):
        assert _norm(**{k: ODD}) == E
    assert _norm(r=P, h=ODD) == E


def _grad(dy=P, h=P, w=P, rstd=P, dh=None, t=F16, wt=F16, rows=4, cols=8, dx=P, dw=P, ws=P, nb=1 << 20):
    return dbf.lib().dbf_rms_norm_backward(dy, h, w, rstd, dh, t, wt, rows, cols, dx, dw, ws, nb, None)


def test_norm_backward_refusals():
    assert _grad(rows=0, dw=None) == dbf.DBF_OK
    for k in ("dy", "h", "rstd"):
        assert _grad(**{k: None}) == E
        assert _grad(**{k: ODD}) == E
    for k in ("w", "dh", "dx", "dw", "ws"):
        assert _grad(**{k: ODD}) == E
    assert _grad(ws=None) == E
    need = dbf.lib().dbf_rms_norm_backward_workspace(4, 8)
    assert need > 0 and _grad(nb=need - 1) == E
    assert _grad(rows=-1) == E
    assert _grad(cols=32769) == dbf.DBF_ERR_SHAPE
    assert _grad(t=E4M3) == E
    assert _grad(wt=BF16) == E
    assert dbf.lib().dbf_rms_norm_backward_workspace(0, 8) == 0


def test_binding_refuses_cpu_tensors_and_bad_formats():
    import torch
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        dbf.mx_quantize(x)
    with pytest.raises(ValueError):
        dbf.mx_quantize(x, "e5m2")
    with pytest.raises(ValueError):
        dbf.MxTensor(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 64, "e4m3")
    with pytest.raises(ValueError):
        dbf.Layer.mx(x)
    with pytest.raises(ValueError):
        dbf.rms_norm(x)
    with pytest.raises(ValueError):
        dbf.rms_norm_backward(x, x, None, torch.zeros(4))


def test_type_constants_match_the_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    names = ["DBF_TYPE_F16", "DBF_TYPE_BF16", "DBF_TYPE_F32", "DBF_TYPE_E4M3", "DBF_TYPE_E2M1"]
    body = "".join(f'    printf("%d\\n", (int){n});\n' for n in names)
    c, exe = str(tmp_path / "t.c"), str(tmp_path / "t")
    open(c, "w").write(f'#include <stdio.h>\n#include "dbf.h"\nint main(void) {{\n{body}    return 0;\n}}\n')
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(root, "include"), c, "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in out] == [getattr(dbf, n) for n in names]
