"""Every tile of the 4-bit layer's products, with K whole and in parts: the host's plan says which sizes reach which,
and on the GPU small whole numbers, whose products and sums are exact, give the bits of the 64-bit result.

Every GPU case prints its name before it touches the GPU.
"""

import ctypes
import sys

import pytest

import dbf_linear_fwd_amd as dbf

E4M3, E2M1 = dbf.DBF_TYPE_E4M3, dbf.DBF_TYPE_E2M1
FMT = {"e4m3": E4M3, "e2m1": E2M1}

# rows, n, m, blocks of x, output type; n a multiple of 8 and odd, m inside a block and at 128 columns, K shorter and
# longer than the pipelines
FORWARD = [
    (19, 209, 207, "e4m3", "f16"), (17, 192, 1280, "e2m1", "bf16"),
    (17, 192, 2351, "e4m3", "bf16"), (17, 217, 2328, "e2m1", "f16"), (17, 217, 4096, "e4m3", "f16"),
    (35, 10329, 201, "e4m3", "bf16"), (64, 4200, 1030, "e2m1", "f16"), (64, 5000, 1030, "e4m3", "f16"),
    (34, 5403, 9146, "e4m3", "f16"), (35, 1432, 8250, "e2m1", "bf16"), (33, 4992, 8996, "e4m3", "bf16"),
    (67, 9669, 200, "e4m3", "f16"), (72, 8648, 1030, "e2m1", "f16"), (72, 8648, 1030, "e4m3", "bf16"),
    (34, 4445, 14293, "e4m3", "bf16"), (68, 3411, 14035, "e2m1", "bf16"),
    (138, 12841, 202, "e4m3", "bf16"), (194, 8899, 1000, "e2m1", "f16"), (130, 14080, 700, "e4m3", "f16"),
    (68, 10896, 13093, "e4m3", "f16"), (85, 11599, 14198, "e2m1", "bf16"),
    (265, 12051, 247, "e4m3", "f16"), (280, 11968, 1300, "e2m1", "bf16"), (280, 11968, 1300, "e4m3", "bf16"),
    (700, 9001, 700, "e2m1", "f16"), (800, 8000, 1300, "e2m1", "bf16"), (500, 11968, 1300, "e4m3", "f16"),
    (226, 10488, 14151, "e4m3", "f16"), (227, 13025, 12571, "e4m3", "bf16"), (800, 4096, 14336, "e4m3", "bf16"),
    (1060, 7445, 201, "e4m3", "bf16"), (1900, 8100, 1030, "e2m1", "f16"), (1900, 8101, 1540, "e4m3", "f16"),
]

# rows, n, m, type; n a multiple of 64, of 8, odd
BACKWARD = [
    (17, 192, 230, "f16"), (18, 208, 208, "bf16"), (19, 209, 207, "f16"),
    (17, 832, 214, "bf16"), (17, 720, 204, "f16"), (17, 725, 208, "bf16"), (77, 4096, 1000, "f16"),
    (195, 192, 10255, "bf16"), (266, 200, 8175, "f16"), (143, 203, 14338, "bf16"), (256, 1024, 14300, "f16"),
    (256, 1000, 14336, "bf16"), (256, 1001, 14336, "f16"),
    (876, 6592, 286, "f16"), (1385, 5240, 261, "bf16"), (97, 7127, 2746, "f16"), (300, 8192, 4096, "bf16"),
    (128, 4096, 8192, "f16"), (512, 14336, 4096, "bf16"),
    (785, 192, 13238, "bf16"), (903, 208, 12226, "f16"), (1556, 203, 7086, "bf16"), (1900, 1024, 8100, "f16"),
    (1000, 14336, 4096, "bf16"), (917, 7352, 8123, "f16"), (211, 14009, 13850, "bf16"), (1900, 14336, 4096, "f16"),
]


def test_forward_sizes_reach_every_tile():
    seen = {}
    for b, n, m, act, _ in FORWARD:
        rows, cols, parts = dbf.dbf_mx_forward_plan(b, n, m, FMT[act])
        seen.setdefault((rows, cols, act), set()).add(parts > 1)
    tiles = [(256, 256), (128, 256), (128, 128), (64, 128), (64, 64), (32, 64)]
    assert set(seen) == {(*t, act) for t in tiles for act in FMT}
    # (the largest tile fills the chip before K is cut; so does the next with the smaller operands)
    whole = {(256, 256, "e4m3"), (256, 256, "e2m1"), (128, 256, "e2m1")}
    assert all(v == ({False} if k in whole else {False, True}) for k, v in seen.items()), seen


def test_backward_sizes_reach_every_tile():
    seen = set()
    for b, n, m, _ in BACKWARD:
        rows, cols, parts = dbf.dbf_mx_backward_plan(b, n, m)
        seen.add((rows, cols, parts > 1, "64" if n % 64 == 0 else "8" if n % 8 == 0 else "odd"))
    assert seen == {(r, c, p, k) for r, c in ((256, 256), (128, 128), (32, 128)) for p in (False, True)
                    for k in ("64", "8", "odd")}


def test_plan_of_few_rows_and_refusals():
    E = dbf.DBF_ERR_INVALID_ARG
    for b in (1, 16):
        assert dbf.dbf_mx_forward_plan(b, 4096, 4096, E4M3) == (0, 0, 1)
    assert dbf.dbf_mx_forward_plan(17, 4096, 4096, E4M3)[0] > 0
    assert dbf.dbf_mx_forward_plan(16, 4096, 14336, E4M3)[0] > 0  # its blocks do not fit one compute unit
    L, plan = dbf.lib(), (ctypes.c_int32 * 3)()
    assert L.dbf_mx_forward_plan(1, 1, 1, E4M3, None) == E and L.dbf_mx_backward_plan(1, 1, 1, None) == E
    for b, n, m in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (-1, 1, 1), (2 ** 31 - 1, 64, 64), (4, 2 ** 31 - 1, 64),
                    (4, 64, 2 ** 31 - 1)):
        assert L.dbf_mx_forward_plan(b, n, m, E4M3, plan) == E and L.dbf_mx_backward_plan(b, n, m, plan) == E
    for t in (dbf.DBF_TYPE_F16, dbf.DBF_TYPE_BF16, dbf.DBF_TYPE_F32, 9):
        assert L.dbf_mx_forward_plan(4, 64, 64, t, plan) == E


# ------------------------------------------------------------------ on the GPU

def _say(msg):
    print(f"[case] {msg}", flush=True)
    sys.stdout.flush()


def _type(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def _weight(gen, n, m):
    """A weight of whole numbers up to 24, half of them zeros, its scales changing from block to block: (MxTensor,
    the numbers in fp64)."""
    import torch
    wide = -(-m // 128) * 128
    c = torch.randint(0, 16, (n, wide), generator=gen, device="cuda")
    c = c * (torch.rand((n, wide), generator=gen, device="cuda") < 0.57)
    c[:, m:] = 0
    s = 128 + torch.randint(0, 2, (n, wide // 32), generator=gen, device="cuda")
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = torch.cat((value, -value))[c] * torch.exp2(s.double() - 127).repeat_interleave(32, dim=1)
    s[:, -(-m // 32):] = 0
    codes = (c[:, 0::2] + 16 * c[:, 1::2]).to(torch.uint8).contiguous()
    return dbf.MxTensor(codes, s.to(torch.uint8).contiguous(), m, "e2m1"), v[:, :m].contiguous()


def _check(got, exact, most):
    """The 64-bit result rounded once to got's type; every sum of magnitudes is a whole number that fp32 holds."""
    import torch
    assert float(most) < 2 ** 24
    assert torch.equal(got, exact.float().to(got.dtype)), int((got != exact.float().to(got.dtype)).sum())


@pytest.mark.gpu
@pytest.mark.parametrize("b,n,m,act,out", FORWARD)
def test_forward_bits(gpu, b, n, m, act, out):
    import torch
    _say(f"mx plan forward b={b} n={n} m={m} {act} {out}")
    gen = torch.Generator(device="cuda").manual_seed(b + n + m)
    W, wv = _weight(gen, n, m)
    if act == "e4m3":  # four significant bits, up to 14: the blocks hold them as they are
        x = torch.randint(-14, 15, (b, m), generator=gen, device="cuda")
    else:              # 0 to 4 and 6, a 4 in every block
        x = torch.randint(-5, 6, (b, m), generator=gen, device="cuda")
        x = torch.where(x.abs() == 5, x.sign() * 6, x)
        x[:, ::32] = 4
    xv = x.double()
    wt = wv.t().contiguous()
    exact, most = torch.mm(xv, wt), torch.mm(xv.abs(), wt.abs()).max()
    L = dbf.Layer.mx(W, max_batch=b, act=act)
    try:
        for rows in ("f16", "bf16"):
            _check(L.forward(x.to(_type(rows)), out_dtype=_type(out)), exact, most)
        _check(L.forward(dbf.mx_quantize(x.half(), act), out_dtype=_type(out)), exact, most)
    finally:
        L.close()


@pytest.mark.gpu
@pytest.mark.parametrize("b,n,m,name", BACKWARD)
def test_backward_bits(gpu, b, n, m, name):
    import torch
    _say(f"mx plan backward b={b} n={n} m={m} {name}")
    gen = torch.Generator(device="cuda").manual_seed(b + n + m)
    W, wv = _weight(gen, n, m)
    dy = torch.randint(-8, 9, (b, n), generator=gen, device="cuda")
    exact, most = torch.mm(dy.double(), wv), torch.mm(dy.double().abs(), wv.abs()).max()
    L = dbf.Layer.mx(W, max_batch=b)
    try:
        d = dy.to(_type(name))
        dx = L.backward_data(d)
        _check(dx, exact, most)
        for _ in range(3):
            assert torch.equal(L.backward_data(d), dx)
    finally:
        L.close()
