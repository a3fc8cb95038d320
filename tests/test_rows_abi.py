"""Argument checks of the entry points of rows in groups, on the host (every call below is refused, or returns,
before any HIP call), and the oracle's own pins."""

import ctypes

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import rows_oracle as O

E, SHAPE, OK, NO = dbf.DBF_ERR_INVALID_ARG, dbf.DBF_ERR_SHAPE, dbf.DBF_OK, dbf.DBF_ERR_UNSUPPORTED
P = ctypes.c_void_p(4096)      # aligned, never dereferenced
ODD = ctypes.c_void_p(4098)
F16, BF16, F32, E4M3, E2M1 = (dbf.DBF_TYPE_F16, dbf.DBF_TYPE_BF16, dbf.DBF_TYPE_F32, dbf.DBF_TYPE_E4M3,
                              dbf.DBF_TYPE_E2M1)
BIG = 1 << 40


def test_group_rows_refusals():
    L = dbf.lib()
    f = lambda index=P, bits=32, rows=5, count=3, order=P, offsets=P, ws=None, nbytes=0: \
        L.dbf_group_rows(index, bits, rows, count, order, offsets, ws, nbytes, None)  # noqa: E731
    assert f(index=None) == E and f(index=ODD) == E and f(order=None) == E and f(order=ODD) == E
    assert f(offsets=None) == E and f(offsets=ODD) == E and f(rows=0, offsets=None) == E
    assert f(index=ctypes.c_void_p(4100), bits=64) == E
    for bits in (0, 16, 33):
        assert f(bits=bits) == E
    assert f(rows=-1) == E and f(count=0) == E and f(count=-4) == E
    assert f(count=1025) == SHAPE and f(rows=(1 << 24) + 1) == SHAPE
    assert f(rows=4097) == E  # no workspace
    need = L.dbf_group_rows_workspace(4097, 3)
    assert need > 0
    assert f(rows=4097, ws=P, nbytes=need - 1) == E and f(rows=4097, ws=ODD, nbytes=need) == E


def test_group_rows_workspace():
    w = dbf.lib().dbf_group_rows_workspace
    assert w(1, 1) == 0 and w(4096, 1024) == 0
    assert w(4097, 1024) == 5 * 1025 * 4 and w(1 << 24, 1) == 1024 * 2 * 4
    for rows, count in ((0, 1), (-1, 1), (5, 0), (5, 1025), ((1 << 24) + 1, 1)):
        assert w(rows, count) == 0


def test_experts_refusals():
    L = dbf.lib()
    h = ctypes.c_void_p()
    H = ctypes.byref(h)
    f = lambda count=2, n=8, m=8, codes=P, scales=P, act=E4M3, rows=4, out=H: \
        L.dbf_experts_pack(count, n, m, codes, scales, act, rows, None, out)  # noqa: E731
    assert f(out=None) == E and f(codes=None) == E and f(scales=None) == E and f(codes=ODD) == E and f(scales=ODD) == E
    for bad in ({"count": 0}, {"n": 0}, {"m": -1}, {"rows": 0}, {"act": F16}):
        assert f(**bad) == E
    for big in ({"count": 1025}, {"n": (1 << 20) + 1}, {"m": (1 << 20) + 1}, {"rows": (1 << 24) + 1},
                {"n": 1 << 20, "m": 1 << 20}, {"m": 1 << 20, "rows": 1 << 20}, {"n": 1 << 20, "rows": 1 << 20}):
        assert f(**big) == SHAPE
    assert h.value is None
    assert L.dbf_experts_forward(None, P, F16, None, P, P, 1, 0, 0, P, F16, None) == E
    assert L.dbf_experts_backward_data(None, P, F16, P, P, 1, 0, 0, P, None) == E


def test_experts_wide_and_many():
    # a launch over every group's tiles stays below 2^32 threads
    pack = dbf.lib().dbf_experts_pack
    out = ctypes.c_void_p()
    for count, n, m in ((1024, 1 << 20, 128), (1024, 128, 1 << 20), (513, 1 << 20, 128), (1024, (1 << 19) + 1, 128)):
        assert pack(count, n, m, P, P, E4M3, 16, None, ctypes.byref(out)) == SHAPE and not out.value


def _adapter(**k):
    a = dict(x=P, base=P, A=P, B=P, scale=P, type=F16, order=P, offsets=P, rows=5, n=8, m=16, rank=4, count=2, y=P, t=P,
             ws=P, nbytes=BIG)
    a.update(k)
    return dbf.lib().dbf_adapter_forward(a["x"], a["base"], a["A"], a["B"], a["scale"], a["type"], a["order"],
                                         a["offsets"], a["rows"], a["n"], a["m"], a["rank"], a["count"], a["y"], a["t"],
                                         a["ws"], a["nbytes"], None)


def _adapter_back(**k):
    Q = ctypes.c_void_p(16384)
    a = dict(dy=P, x=P, t=P, dx=Q, A=P, B=P, scale=P, type=F16, order=P, offsets=P, rows=5, n=8, m=16, rank=4, count=2,
             out=Q, dA=P, dB=P, ws=P, nbytes=BIG)
    a.update(k)
    return dbf.lib().dbf_adapter_backward(a["dy"], a["x"], a["t"], a["dx"], a["A"], a["B"], a["scale"], a["type"],
                                          a["order"], a["offsets"], a["rows"], a["n"], a["m"], a["rank"], a["count"],
                                          a["out"], a["dA"], a["dB"], a["ws"], a["nbytes"], None)


SIZES = [({"rows": -1}, E), ({"n": 0}, E), ({"m": 0}, E), ({"rank": 0}, E), ({"count": 0}, E), ({"type": F32}, E),
         ({"type": E4M3}, E), ({"rank": 129}, SHAPE), ({"count": 1025}, SHAPE), ({"n": (1 << 18) + 1}, SHAPE),
         ({"m": (1 << 18) + 1}, SHAPE), ({"rows": (1 << 24) + 1}, SHAPE),
         ({"rows": 1 << 24, "n": 1 << 13}, SHAPE), ({"count": 1024, "rank": 128, "m": 1 << 16}, SHAPE)]


@pytest.mark.parametrize("bad,status", SIZES)
def test_adapter_sizes(bad, status):
    assert _adapter(**bad) == status and _adapter_back(**bad) == status


def test_adapter_refusals():
    for k in ("x", "base", "A", "B", "y", "ws", "order", "offsets"):
        assert _adapter(**{k: None}) == E and _adapter(**{k: ODD}) == E
    for k in ("scale", "t"):
        assert _adapter(**{k: ODD}) == E
    L = dbf.lib()
    need = L.dbf_adapter_workspace(5, 8, 16, 4, 2)
    assert need > 0 and _adapter(nbytes=need - 1) == E
    assert _adapter(rows=0) == OK and _adapter(rows=0, x=None, order=None, ws=None) == OK
    assert L.dbf_adapter_workspace(0, 8, 16, 4, 2) == 0 and L.dbf_adapter_workspace(5, 8, 16, 129, 2) == 0


def test_adapter_backward_refusals():
    for k in ("dy", "A", "B", "ws", "order", "offsets", "x", "t"):
        assert _adapter_back(**{k: None}) == E
    for k in ("dy", "x", "t", "dx", "A", "B", "ws", "order", "offsets", "scale", "out", "dA", "dB"):
        assert _adapter_back(**{k: ODD}) == E
    L = dbf.lib()
    need = L.dbf_adapter_backward_workspace(5, 8, 16, 4, 2)
    assert need > 0 and _adapter_back(nbytes=need - 1) == E
    assert _adapter_back(out=None, dA=None, dB=None) == OK  # nothing to compute
    other = ctypes.c_void_p(8192)
    assert _adapter_back(x=other, out=other) == E and _adapter_back(dy=other, out=other) == E
    assert _adapter_back(rows=0, dA=None, dB=None) == OK
    assert L.dbf_adapter_backward_workspace(0, 8, 16, 4, 2) == 0


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError):
        dbf.group_rows(torch.zeros(4, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        dbf.RowGroups(torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError):
        dbf.Adapters(torch.zeros(1, 2, 8, dtype=torch.float16), torch.zeros(1, 8, 2, dtype=torch.float16))
    with pytest.raises(ValueError):
        dbf.Experts(torch.zeros(4, 4), 2, 4)


def test_oracle_group_rows_by_hand():
    order, offsets = O.group_rows([2, 0, -1, 2, 1, 5, 0], 3)
    assert order.tolist() == [1, 6, 4, 0, 3, 2, 5] and offsets.tolist() == [0, 2, 3, 5]
    assert O.places(order, offsets).tolist() == [0, 0, 1, 2, 2, 3, 3]


def test_oracle_experts_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])  # two tokens, two experts each; token 1's second is none
    w = [np.array([[1.0, 0.0]]), np.array([[0.0, 10.0]])]
    order, offsets = O.group_rows([1, 0, 0, -1], 2)
    assert O.experts(x, w, order, offsets, 2, False)[:, 0].tolist() == [1.0, 3.0, 20.0, 0.0]
    assert O.experts(x, w, order, offsets, 2, True)[:, 0].tolist() == [20.0, 1.0, 3.0, 0.0]


def test_oracle_adapter_gradients_are_differences():
    rng = np.random.default_rng(5)
    rows, n, m, r, count = 6, 4, 5, 3, 2
    index = [0, 1, -1, 0, 1, 1]
    x, dy = rng.standard_normal((rows, m)), rng.standard_normal((rows, n))
    A, B, s = rng.standard_normal((count, r, m)), rng.standard_normal((count, n, r)), rng.standard_normal(count)
    loss = lambda x, A, B: (O.adapters(x, np.zeros((rows, n)), A, B, s, index)[0] * dy).sum()  # noqa: E731
    t = O.adapters(x, np.zeros((rows, n)), A, B, s, index)[1]
    dx, _, dA, dB = O.adapters_backward(dy, x, t, np.zeros((rows, m)), A, B, s, index)
    h = 1e-6
    for k, grad in ((0, dx), (1, dA), (2, dB)):
        v = [x, A, B]
        for at in np.ndindex(v[k].shape):
            up, down = [a.copy() for a in v], [a.copy() for a in v]
            up[k][at] += h
            down[k][at] -= h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - grad[at]) < 1e-7
