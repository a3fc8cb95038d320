"""GPU: bf16 adapters whose t and u are finite in fp32 and above bf16's largest value: 2^128 - 2^118 and its negative.

The first of their 16-bit parts is bf16's largest value then, 2^128 - 2^120, and
the second holds the rest, so results that fit are off by what the parts
always lose (2^-17 of t in y and dx', 2^-25 in dA and dB), the sums (at most
64 roundings of 2^-24) and the result's own rounding, and a zero of the other
factor stays a zero.

Every case prints its name before it touches the GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf

pytestmark = pytest.mark.gpu

EDGE = 2.0 ** 128 - 2.0 ** 118
TOP, REST = 2.0 ** 128 - 2.0 ** 120, 1.5 * 2.0 ** 119  # bf16 values, together EDGE


def _bf16(v):
    import torch
    return torch.from_numpy(np.ascontiguousarray(v, dtype=np.float64)).to(torch.bfloat16).cuda()


def _within(got, ref, rel):
    got = got.double().cpu().numpy()
    assert np.all(np.abs(got - ref) <= rel * np.abs(ref)), (got[np.abs(got - ref) > rel * np.abs(ref)][:4], got.shape)


# rows, width: one row tile, and several
@pytest.mark.parametrize("rows,width", [(3, 72), (600, 7200)])
@pytest.mark.parametrize("rank", [2, 24, 64, 100])
def test_largest_t(gpu, rows, width, rank):
    import torch
    print(f"[case] largest t: {rows} rows, {width} columns, rank {rank}", flush=True)
    rng = np.random.default_rng(rank)
    sign = rng.choice([-1.0, 1.0], rows)
    x = np.zeros((rows, 8))
    x[:, 0], x[:, 1], x[:, 2] = sign * TOP, sign * REST, 1.0
    A = np.zeros((1, rank, 8))
    A[0, 0, :2] = 1.0   # t[0] = +-EDGE
    A[0, 1, 2] = 1.0    # t[1] = 1
    B = np.zeros((1, width, rank))
    B[0, :, 0] = 2.0 ** -10 * rng.integers(-3, 4, width)
    B[0, B[0, :, 0] == 0, 1] = 5.0
    base = np.zeros((rows, width))
    g = dbf.group_rows(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1)
    y, t = dbf.Adapters(_bf16(A), _bf16(B))(_bf16(x), _bf16(base), g)
    tv = t.double().cpu().numpy()
    assert np.array_equal(tv[:, 0], sign * EDGE) and np.all(tv[:, 1] == 1.0)
    _within(y, tv @ B[0].T, 2.0 ** -8 + 2.0 ** -16 + 64 * 2.0 ** -24)


@pytest.mark.parametrize("rows,width", [(3, 72), (600, 7200)])
@pytest.mark.parametrize("rank", [2, 24, 64, 100])
def test_largest_u(gpu, rows, width, rank):
    """dx' and dA at u = +-EDGE, dB at such a t."""
    import torch
    print(f"[case] largest u: {rows} rows, {width} columns, rank {rank}", flush=True)
    rng = np.random.default_rng(rank)
    sign = rng.choice([-1.0, 1.0], rows)
    dy = np.zeros((rows, 8))
    dy[:, 0], dy[:, 1], dy[:, 2] = sign * TOP, sign * REST, 1.0
    B = np.zeros((1, 8, rank))
    B[0, :2, 0] = 1.0
    B[0, 2, 1] = 1.0
    A = np.zeros((1, rank, width))
    A[0, 0] = 2.0 ** -10 * rng.integers(-3, 4, width)
    A[0, 1, A[0, 0] == 0] = 5.0
    # the gradients' sums: of one row, the others are zeros
    x = np.zeros((rows, width))
    x[1] = 2.0 ** -10 * rng.integers(-3, 4, width)
    t = np.zeros((rows, rank))
    t[2, 0], t[2, 1] = EDGE, 1.0
    dy[2] = 2.0 ** -10
    g = dbf.group_rows(torch.zeros(rows, dtype=torch.int32, device="cuda"), 1)
    dx, dA, dB = dbf.Adapters(_bf16(A), _bf16(B)).backward(_bf16(dy), _bf16(x),
                                                           torch.from_numpy(t).float().cuda(), g)
    u = dy @ B[0]
    assert u[1, 0] == sign[1] * EDGE
    _within(dx, u @ A[0], 2.0 ** -8 + 2.0 ** -16 + 64 * 2.0 ** -24)
    _within(dA[0], u.T @ x, 2.0 ** -24 + 64 * 2.0 ** -24)
    # (row 2 alone has t)
    _within(dB[0], dy.T @ t, 2.0 ** -24 + 64 * 2.0 ** -24)
