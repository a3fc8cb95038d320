"""Every tile of the experts' products and gradients, with the sum whole and in parts: the host's plan and the groups'
sizes say which case reaches which, and on the GPU small whole numbers, whose products and sums are exact, give the
bits of the 64-bit result.

In the tiles of eight waves some have no rows where a group ends in the lower
half of a tile; their cases have groups that end in either half.  Cases of
more than 64 experts take their row tiles from a table.

Every GPU case prints its name before it touches the GPU.
"""

import ctypes

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from tests import test_mx_plans as P

FMT = P.FMT

# experts, n, m, tokens, experts of a token, blocks of x, output type; the last three are one token, a decode batch
# and a prompt of 4-bit experts at their usual widths
FORWARD = [
    (1, 64, 68, 2, 4, "e4m3", "f16"), (1, 72, 74, 4, 3, "e2m1", "bf16"), (65, 66, 64, 63, 3, "e4m3", "bf16"),
    (65, 72, 65, 9, 4, "e2m1", "f16"), (1, 64, 3718, 2, 3, "e4m3", "bf16"), (1, 79, 3584, 3, 4, "e2m1", "f16"),
    (65, 71, 4546, 11, 2, "e4m3", "f16"), (65, 64, 7141, 40, 2, "e2m1", "bf16"),
    (2, 77, 65, 1859, 3, "e4m3", "bf16"), (13, 70, 75, 2216, 3, "e2m1", "f16"), (80, 66, 65, 1264, 4, "e4m3", "f16"),
    (65, 80, 68, 2080, 2, "e2m1", "bf16"), (1, 67, 4888, 178, 4, "e4m3", "f16"), (1, 76, 4864, 215, 3, "e2m1", "f16"),
    (65, 64, 12629, 733, 4, "e4m3", "bf16"), (65, 64, 9917, 716, 4, "e2m1", "bf16"),
    (8, 72, 71, 9363, 2, "e4m3", "f16"), (13, 72, 133, 3964, 4, "e2m1", "bf16"), (128, 68, 79, 4883, 3, "e4m3", "bf16"),
    (65, 76, 130, 4823, 3, "e2m1", "f16"), (8, 74, 7615, 375, 4, "e4m3", "bf16"), (2, 68, 8581, 629, 3, "e2m1", "f16"),
    (40, 86, 64, 11629, 2, "e4m3", "f16"), (13, 72, 70, 10088, 2, "e2m1", "bf16"), (128, 65, 74, 5097, 4, "e4m3", "bf16"),
    (65, 75, 66, 10707, 2, "e2m1", "f16"), (3, 67, 13874, 614, 4, "e4m3", "f16"), (3, 163, 7143, 7397, 4, "e2m1", "bf16"),
    (3, 140, 5888, 5447, 4, "e4m3", "bf16"), (8, 216, 14167, 4745, 4, "e2m1", "f16"), (128, 144, 6456, 3334, 4, "e4m3", "f16"),
    (80, 184, 14146, 6797, 2, "e2m1", "bf16"),
    (64, 672, 65, 5809, 2, "e4m3", "f16"), (5, 323, 68, 9332, 3, "e2m1", "bf16"), (65, 385, 76, 5965, 3, "e4m3", "bf16"),
    (100, 448, 72, 6948, 2, "e2m1", "f16"), (2, 3584, 919, 4635, 2, "e4m3", "bf16"), (3, 1562, 1024, 13928, 2, "e4m3", "f16"),
    (3, 6336, 983, 2516, 3, "e2m1", "f16"), (3, 1562, 1024, 13928, 2, "e2m1", "bf16"), (65, 1698, 1755, 9658, 3, "e4m3", "f16"),
    (65, 3104, 1112, 8756, 3, "e2m1", "bf16"),
    (3, 9240, 409, 4554, 4, "e4m3", "bf16"), (1, 655, 4561, 11544, 2, "e4m3", "f16"), (3, 1344, 1223, 6972, 3, "e2m1", "f16"),
    (8, 14336, 4096, 1, 2, "e4m3", "f16"), (64, 4096, 1024, 16, 8, "e4m3", "bf16"), (8, 14336, 4096, 2048, 2, "e4m3", "bf16"),
    (8, 14336, 4096, 2047, 2, "e2m1", "f16"),
]

# experts, n, m, tokens, experts of a token, type; n a multiple of 64, of 8, others (whose rows are padded)
BACKWARD = [
    (1, 64, 68, 2, 4, "f16"), (1, 72, 85, 5, 2, "bf16"), (1, 73, 78, 6, 2, "f16"), (65, 72, 65, 9, 4, "bf16"),
    (1, 832, 71, 3, 3, "bf16"), (1, 736, 66, 4, 2, "f16"), (1, 783, 78, 3, 3, "bf16"), (65, 836, 65, 10, 3, "f16"),
    (1, 64, 138, 2983, 4, "bf16"), (8, 72, 67, 11204, 2, "f16"), (2, 65, 66, 8496, 3, "bf16"), (65, 75, 66, 10707, 2, "f16"),
    (2, 8384, 73, 674, 3, "f16"), (1, 6808, 140, 575, 2, "bf16"), (2, 8245, 130, 371, 3, "f16"), (80, 5353, 66, 1858, 4, "bf16"),
    (65, 5784, 68, 1785, 4, "f16"),
    (64, 64, 513, 4787, 2, "bf16"), (100, 96, 134, 14521, 2, "f16"), (80, 65, 710, 5147, 1, "bf16"), (5, 66, 11520, 85, 4, "f16"),
    (128, 64, 160, 9426, 3, "bf16"), (2, 7360, 131, 713, 4, "f16"), (2, 8128, 167, 1146, 3, "bf16"),
    (2, 8560, 155, 1380, 2, "bf16"), (2, 10344, 672, 211, 4, "f16"), (3, 8858, 166, 1347, 2, "bf16"), (2, 9019, 156, 1314, 2, "f16"),
    (100, 582, 1280, 6089, 4, "bf16"), (65, 696, 939, 12023, 2, "f16"),
    (8, 14336, 4096, 1, 2, "f16"), (64, 4096, 1024, 16, 8, "bf16"), (8, 14336, 4096, 2048, 2, "bf16"),
]


def group_sizes(count, slots):
    """Uneven groups, one of them without rows where there are more than three, and some rows of none."""
    part = np.random.default_rng(count * 1000003 + slots).random(count + 1) ** 2 + 0.02
    part[count] *= 0.3
    if count > 3:
        part[count // 2] = 0
    return [int(v) for v in (slots * part / part.sum()).astype(int)[:count]]


def parts_of(plan, sizes, cols, steps):
    """(K parts of the cut tiles, how groups end in a tile: in its lower half, in its upper half)."""
    rows, width, most, room, _ = plan
    rest = sum(-(-s // rows) for s in sizes) * -(-cols // width) % room
    parts = min(room // rest, most, steps // 4) if rest else 1
    ends = {(s % rows) > rows // 2 for s in sizes if s % rows}
    return max(parts, 1), ends


def test_forward_sizes_reach_every_tile():
    seen, table, placed, ends = {}, set(), set(), {}
    for count, n, m, tokens, top, act, _ in FORWARD:
        slots = tokens * top
        plan = dbf.dbf_experts_forward_plan(count, n, m, slots, FMT[act])
        parts, e = parts_of(plan, group_sizes(count, slots), n, -(-m // 128))
        seen.setdefault((plan[0], plan[1], act), set()).add(parts > 1)
        ends.setdefault((plan[0], plan[1], act, parts > 1), set()).update(e)
        if count > 64:
            table.add((plan[0], plan[1], parts > 1, act))
        if plan[4]:
            placed.add((act, top > 1, slots % 32 > 0))
    tiles = [(256, 256), (128, 256), (128, 128), (64, 128), (64, 64), (32, 64)]
    assert set(seen) == {(*t, act) for t in tiles for act in FMT}
    # (a tile of this width, or of e2m1, has its best sizes where the sum is short)
    whole = {(128, 256, "e4m3"), (128, 256, "e2m1"), (128, 128, "e2m1")}
    assert all(v == ({False} if k in whole else {False, True}) for k, v in seen.items()), seen
    for k, v in ends.items():
        if k[1] == 256:
            assert v == {False, True}, k
    assert {(32, 64, True), (64, 64, True), (256, 256, True)} | {(*t, False) for t in tiles} <= {t[:3] for t in table}
    assert {(act, True, True) for act in FMT} <= placed


def test_backward_sizes_reach_every_tile():
    seen, table, ends = set(), set(), {}
    for count, n, m, tokens, top, _ in BACKWARD:
        slots = tokens * top
        plan = dbf.dbf_experts_backward_plan(count, n, m, slots)
        parts, e = parts_of(plan, group_sizes(count, slots), m, -(-n // 64))
        seen.add((plan[0], plan[1], parts > 1, "64" if n % 64 == 0 else "8" if n % 8 == 0 else "other"))
        ends.setdefault((plan[0], parts > 1), set()).update(e)
        if count > 64:
            table.add((plan[0], plan[1], parts > 1))
    tiles = {(r, c, p) for r, c in ((256, 256), (128, 128), (32, 128)) for p in (False, True)}
    assert {(*t, k) for t in tiles for k in ("64", "8", "other")} <= seen, {(*t, k) for t in tiles for k in ("64", "8", "other")} - seen
    assert table == tiles and ends[256, False] == ends[256, True] == {False, True}


def test_plans_and_refusals():
    E, SHAPE = dbf.DBF_ERR_INVALID_ARG, dbf.DBF_ERR_SHAPE
    L, plan = dbf.lib(), (ctypes.c_int32 * 5)()
    f = lambda count=2, n=64, m=64, slots=4, x_type=dbf.DBF_TYPE_E4M3, out=plan: \
        L.dbf_experts_forward_plan(count, n, m, slots, x_type, out)  # noqa: E731
    b = lambda count=2, n=64, m=64, slots=4, out=plan: L.dbf_experts_backward_plan(count, n, m, slots, out)  # noqa: E731
    assert f() == 0 and b() == 0
    for bad in ({"count": 0}, {"n": 0}, {"m": -1}, {"slots": 0}, {"out": None}):
        assert f(**bad) == E and b(**bad) == E
    for t in (dbf.DBF_TYPE_F16, dbf.DBF_TYPE_BF16, dbf.DBF_TYPE_F32, 9):
        assert f(x_type=t) == E
    for big in ({"count": 1025}, {"n": (1 << 20) + 1}, {"m": (1 << 20) + 1}, {"slots": (1 << 24) + 1},
                {"n": 1 << 20, "m": 1 << 20}, {"m": 1 << 20, "slots": 1 << 20}, {"n": 1 << 20, "slots": 1 << 20},
                {"count": 513, "n": 1 << 20}):
        assert f(**big) == SHAPE and b(**big) == SHAPE
    # parts of a round at most, and none of a short sum
    assert dbf.dbf_experts_forward_plan(8, 14336, 128, 64, dbf.DBF_TYPE_E4M3)[2] == 1
    assert dbf.dbf_experts_backward_plan(8, 64, 14336, 64)[2] == 1
    assert dbf.dbf_experts_backward_plan(3, 65, 64, 8)[4] == 1 and dbf.dbf_experts_backward_plan(3, 64, 65, 8)[4] == 0


# ------------------------------------------------------------------ on the GPU

def _routes(count, slots, gen):
    """(index, grouped order's RowGroups) with the sizes of group_sizes, in a random order."""
    import torch
    sizes = group_sizes(count, slots)
    index = torch.full((slots,), -1, dtype=torch.int32)
    index[:sum(sizes)] = torch.repeat_interleave(torch.arange(count, dtype=torch.int32), torch.tensor(sizes))
    index = index.cuda()[torch.randperm(slots, generator=gen, device="cuda")].contiguous()
    return index, dbf.group_rows(index, count)


def _exact(rows, w, index, count):
    """The 64-bit result of every slot (rows: one for each), and the largest sum of magnitudes."""
    import torch
    out, most = torch.zeros(rows.shape[0], w[0].shape[0], dtype=torch.float64, device="cuda"), 0.0
    for e in range(count):
        at = torch.nonzero(index == e).flatten()
        if at.numel():
            x, wt = rows[at].double(), w[e].t().contiguous()
            out[at] = torch.mm(x, wt)
            most = max(most, float(torch.mm(x.abs(), wt.abs()).max()))
    return out, most


def _weights(gen, count, n, m):
    W, v = P._weight(gen, count * n, m)
    return W, v.view(count, n, m)


@pytest.mark.gpu
@pytest.mark.parametrize("count,n,m,tokens,top,act,out", FORWARD)
def test_forward_bits(gpu, count, n, m, tokens, top, act, out):
    import torch
    P._say(f"experts plan forward {count} x {n} x {m}, {tokens} tokens x {top}, {act} {out}")
    gen = torch.Generator(device="cuda").manual_seed(count + n + m)
    W, w = _weights(gen, count, n, m)
    slots = tokens * top
    index, g = _routes(count, slots, gen)
    order = g.order.long()
    if act == "e4m3":  # four significant bits, up to 14: the blocks hold them as they are
        x = torch.randint(-14, 15, (tokens, m), generator=gen, device="cuda")
    else:              # 0 to 4 and 6, a 4 in every block
        x = torch.randint(-5, 6, (tokens, m), generator=gen, device="cuda")
        x = torch.where(x.abs() == 5, x.sign() * 6, x)
        x[:, ::32] = 4
    exact, most = _exact(x.repeat_interleave(top, dim=0), w, index, count)
    assert most < 2 ** 24
    want = exact.float().to(P._type(out))
    ex = dbf.Experts(W, count, slots, act=act)
    try:
        xd = x.to(P._type(out))
        assert torch.equal(ex.forward(xd, g, gather=top), want[order])
        assert torch.equal(ex.forward(dbf.mx_quantize(xd, act), g, gather=top, scatter=True, out_dtype=P._type(out)), want)
        by_place = xd.repeat_interleave(top, dim=0)[order].contiguous()
        assert torch.equal(ex.forward(by_place, g, scatter=True), want)
        assert torch.equal(ex.forward(dbf.mx_quantize(by_place, act), g, out_dtype=P._type(out)), want[order])
    finally:
        ex.close()


@pytest.mark.gpu
@pytest.mark.parametrize("count,n,m,tokens,top,name", BACKWARD)
def test_backward_bits(gpu, count, n, m, tokens, top, name):
    import torch
    P._say(f"experts plan backward {count} x {n} x {m}, {tokens} tokens x {top}, {name}")
    gen = torch.Generator(device="cuda").manual_seed(count + n + m)
    W, w = _weights(gen, count, n, m)
    slots = tokens * top
    index, g = _routes(count, slots, gen)
    order = g.order.long()
    dy = torch.randint(-8, 9, (tokens, n), generator=gen, device="cuda")
    exact, most = _exact(dy.repeat_interleave(top, dim=0), w.transpose(1, 2), index, count)
    assert most < 2 ** 24
    want = exact.float().to(P._type(name))
    ex = dbf.Experts(W, count, slots)
    try:
        d = dy.to(P._type(name))
        assert torch.equal(ex.backward_data(d, g, gather=top), want[order])
        by_place = d.repeat_interleave(top, dim=0)[order].contiguous()
        assert torch.equal(ex.backward_data(by_place, g, scatter=True), want)
        for _ in range(2):
            assert torch.equal(ex.backward_data(d, g, gather=top, scatter=True), want)
    finally:
        ex.close()
