"""GPU: the grouped order of rows, against the oracle: whole numbers, equal.

Every case prints its name before it touches the GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import rows_oracle as O

pytestmark = pytest.mark.gpu


def _say(msg):
    print(f"[case] {msg}", flush=True)


def _torch():
    import torch
    return torch


def same(index, count, dtype):
    torch = _torch()
    g = dbf.group_rows(torch.from_numpy(np.asarray(index, np.int64)).to(dtype).cuda(), count)
    order, offsets = O.group_rows(index, count)
    assert g.order.dtype == torch.int32 and g.offsets.dtype == torch.int32
    assert g.rows == len(index) and g.count == count
    assert np.array_equal(g.offsets.cpu().numpy(), offsets)
    assert np.array_equal(g.order.cpu().numpy(), order)


@pytest.mark.parametrize("bits", [32, 64])
@pytest.mark.parametrize("count", [1, 2, 7, 64, 1000, 1024])
@pytest.mark.parametrize("rows", [0, 1, 2, 63, 64, 65, 128, 1000, 1025, 2048, 2049, 4096, 4097, 16385, 32768, 32769, 131072, 131073])
def test_order(gpu, rows, count, bits):
    _say(f"group_rows {rows} rows {count} groups int{bits}")
    rng = np.random.default_rng(rows + count)
    index = rng.integers(-1, count + 1, size=rows)  # count: of no group, as -1 is
    same(index, count, _torch().int64 if bits == 64 else _torch().int32)


def test_a_million_rows(gpu):
    """More workgroups than add up each other's counts."""
    torch = _torch()
    for rows, count in ((1 << 20, 64), ((1 << 20) + 1, 1000), (3_000_001, 7)):
        _say(f"group_rows {rows} rows {count} groups")
        index = torch.randint(-1, count, (rows,), dtype=torch.int32, device="cuda")
        g = dbf.group_rows(index, count)
        key = torch.where(index < 0, count, index)
        order = torch.sort(key, stable=True).indices
        assert torch.equal(g.order, order.int())
        assert torch.equal(g.offsets, torch.bincount(key, minlength=count + 1).cumsum(0)[:count + 1].int()
                           - torch.bincount(key, minlength=count + 1)[:count + 1].int())


@pytest.mark.parametrize("rows", [70, 20000])
def test_extremes(gpu, rows):
    _say(f"group_rows extremes {rows}")
    torch = _torch()
    for value in (0, 4, -1, 5, 2 ** 31 - 1, -2 ** 31):
        same(np.full(rows, value), 5, torch.int32)
    for value in (2 ** 32, 2 ** 32 + 3, -2 ** 63, 2 ** 63 - 1):  # 64 bits are not cut to 32
        same(np.full(rows, value, dtype=np.int64), 5, torch.int64)
    same(np.arange(rows) % 5, 5, torch.int32)
    same(np.arange(rows)[::-1] * 5 // rows, 5, torch.int32)


def test_empty_and_skewed_groups(gpu):
    _say("group_rows skewed")
    rng = np.random.default_rng(3)
    index = np.where(rng.random(9000) < 0.9, 700, rng.integers(0, 1024, 9000))
    same(index, 1024, _torch().int32)


def test_refusals(gpu):
    torch = _torch()
    ok = torch.zeros(8, dtype=torch.int32, device="cuda")
    for bad in (ok.float(), ok[::2], ok.view(2, 4), ok.to(torch.int16)):
        with pytest.raises(ValueError):
            dbf.group_rows(bad, 2)
    for count in (0, -1, 1025):
        with pytest.raises(ValueError):
            dbf.group_rows(ok, count)


@pytest.mark.parametrize("rows", [500, 40000])
def test_captured_and_on_another_stream(gpu, rows):
    _say(f"group_rows captured {rows}")
    torch = _torch()
    rng = np.random.default_rng(rows)
    index = torch.empty(rows, dtype=torch.int32, device="cuda")
    first = torch.from_numpy(rng.integers(-1, 9, rows)).to(torch.int32)
    index.copy_(first)
    dbf.group_rows(index, 9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = dbf.group_rows(index, 9)
    side.synchronize()
    order, offsets = O.group_rows(first.numpy(), 9)
    assert np.array_equal(g.order.cpu().numpy(), order) and np.array_equal(g.offsets.cpu().numpy(), offsets)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = dbf.group_rows(index, 9)
    for seed in range(3):
        v = np.random.default_rng(100 + seed).integers(-1, 9, rows)
        index.copy_(torch.from_numpy(v).to(torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        order, offsets = O.group_rows(v, 9)
        assert np.array_equal(g.order.cpu().numpy(), order) and np.array_equal(g.offsets.cpu().numpy(), offsets)
        (torch.ones(1000, device="cuda") * 2).sum().item()  # the program's own work between replays
