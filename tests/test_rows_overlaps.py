"""Results over rows that are still read are refused: adapters on the host (before any HIP call), experts on the GPU
(the handle is there); results beside them, or over rows that have been read, are not."""

import ctypes

import pytest

import dbf_linear_fwd_amd as dbf

E, OK = dbf.DBF_ERR_INVALID_ARG, dbf.DBF_OK
BIG = 1 << 40
ROWS, N, M = 8, 16, 32  # bytes: 256 of base and dy, 512 of x and dx


def _p(at):
    return ctypes.c_void_p(at) if at else None


def _forward(base, y):
    P = _p(1 << 16)
    return dbf.lib().dbf_adapter_forward(P, _p(base), P, P, None, dbf.DBF_TYPE_F16, P, P, ROWS, N, M, 4, 2, _p(y), None, P,
                                         BIG, None)


def _backward(dy, x, dx, out):
    P = _p(1 << 16)
    return dbf.lib().dbf_adapter_backward(_p(dy), _p(x), P, _p(dx), P, P, None, dbf.DBF_TYPE_F16, P, P, ROWS, N, M, 4, 2,
                                          _p(out), P, P, P, BIG, None)


def test_adapters_on_the_host():
    base = 1 << 20
    for shift in (16, 128, 240, -16, -240):
        assert _forward(base, base + shift) == E
    dy, x, dx = 1 << 20, 1 << 21, 1 << 22
    for out in (dy, dy + 240, dy - 496, x, x + 16, x + 496, x - 496, dx + 16, dx + 496, dx - 16):
        assert _backward(dy, x, dx, out) == E, out


@pytest.mark.gpu
def test_adapters_beside(gpu):
    """Neighbours, in place, and y over an x that has been read."""
    import torch
    rows, n, rank = 40, 64, 8
    gen = torch.Generator(device="cuda").manual_seed(1)
    A, B = (torch.randn(2, *s, generator=gen, device="cuda").half() for s in ((rank, n), (n, rank)))
    ad = dbf.Adapters(A, B)
    g = dbf.group_rows(torch.randint(-1, 2, (rows,), generator=gen, device="cuda", dtype=torch.int32), 2)
    room = torch.randn(3 * rows, n, generator=gen, device="cuda").half()
    x, base, y = room[:rows], room[rows:2 * rows], room[2 * rows:]
    want, t = ad(x.clone(), base.clone(), g)
    assert torch.equal(ad(x, base, g, out=y).y, want)
    keep = x.clone()
    assert torch.equal(ad(x, base, g, out=x).y, want)
    x.copy_(keep)
    assert torch.equal(ad(x, base, g, out=base).y, want)
    dy, dx = room[rows:2 * rows], room[2 * rows:]
    ref = ad.backward(dy.clone(), x.clone(), t, g, dx=dx.clone())
    got = ad.backward(dy, x, t, g, dx=dx, out=dx)
    assert all(torch.equal(p, q) for p, q in zip(got, ref))
    for out in (room[1:rows + 1], room[rows - 1:2 * rows - 1], room[rows + 1:2 * rows + 1]):
        with pytest.raises(dbf.DbfError):
            ad.backward(dy, x, t, g, out=out)
    for out in (room[rows + 1:2 * rows + 1], room[2 * rows - 1:3 * rows - 1]):
        with pytest.raises(dbf.DbfError):
            ad(x, base, g, out=out)


@pytest.mark.gpu
def test_experts(gpu):
    import torch
    count, n, slots = 3, 128, 50
    gen = torch.Generator(device="cuda").manual_seed(2)
    W = dbf.mx_quantize(torch.randn(count * n, n, generator=gen, device="cuda"), "e2m1")
    ex = dbf.Experts(W, count, slots)
    g = dbf.group_rows(torch.randint(-1, count, (slots,), generator=gen, device="cuda", dtype=torch.int32), count)
    room = torch.randn(3 * slots, n, generator=gen, device="cuda").half()
    x, dy = room[:slots], room[slots:2 * slots]
    # gradients: over dy, over a part of it, beside it
    want = ex.backward_data(dy.clone(), g)
    for out in (dy, room[slots - 1:2 * slots - 1], room[2 * slots - 1:3 * slots - 1]):
        with pytest.raises(dbf.DbfError):
            ex.backward_data(dy, g, out=out)
    assert torch.equal(ex.backward_data(dy, g, out=room[2 * slots:]), want)
    # ready blocks: codes and scales
    q = dbf.mx_quantize(x, "e4m3")
    y = ex.forward(q, g)
    store = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    codes, scales = store[:q.codes.numel()], store[1 << 15:(1 << 15) + q.scales.numel()]
    codes.copy_(q.codes.flatten())
    scales.copy_(q.scales.flatten())
    inside = dbf.MxTensor(codes.view(q.codes.shape), scales.view(q.scales.shape), n, "e4m3")
    for at in (0, codes.numel() - 16, (1 << 15) + scales.numel() - 8, (1 << 15) - 2 * slots * n + 16):
        out = store[at // 16 * 16:][:2 * slots * n].view(torch.float16).view(slots, n)
        with pytest.raises(dbf.DbfError):
            ex.forward(inside, g, out=out)
    out = store[1 << 14:(1 << 14) + 2 * slots * n].view(torch.float16).view(slots, n)
    assert codes.numel() <= 1 << 14 and (1 << 14) + 2 * slots * n <= 1 << 15
    assert torch.equal(ex.forward(inside, g, out=out), y)
    # 16-bit rows are quantised before: a result over them has the same bits
    want = ex(x.clone(), g)
    assert torch.equal(ex(x, g, out=x), want)
    ex.close()
