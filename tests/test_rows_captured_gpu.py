"""GPU: captured calls on rows in groups at the sizes of prompts: the sort in several launches, experts whose products are
cut, take a table of row tiles or put block scales by place, and adapters of several row tiles; replayed on other routes
and rows, with eager work between, equal to the eager calls bit for bit.

Every case prints its name before it touches the GPU.
"""

import pytest

import dbf_linear_fwd_amd as dbf
from tests import test_experts_plans as E

pytestmark = pytest.mark.gpu


def _index(torch, gen, slots, count):
    """Routes of another spread each time, some of none."""
    weight = torch.rand(count, generator=gen, device="cuda") ** 3 + 0.01
    index = torch.multinomial(weight, slots, replacement=True, generator=gen).to(torch.int32)
    index[torch.rand(slots, generator=gen, device="cuda") < 0.1] = -1
    return index


def _replays(torch, step, fill):
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(4):
        fill(torch.Generator(device="cuda").manual_seed(seed))
        graph.replay()
        copies = [v.clone() for v in got]
        torch.cuda.synchronize()
        want = step()
        for a, b in zip(copies, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("count,n,m,tokens,top,act", [
    (3, 6336, 983, 2516, 3, "e2m1"), (65, 1698, 1755, 9658, 3, "e4m3"), (3, 1344, 1223, 6972, 3, "e2m1"),
    (100, 582, 1280, 6089, 4, "e4m3"), (2, 8245, 130, 371, 3, "e4m3")])
def test_experts(gpu, count, n, m, tokens, top, act):
    import torch
    print(f"[case] captured experts {count} x {n} x {m}, {tokens} tokens x {top}, {act}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(1)
    W, _ = E._weights(gen, count, n, m)
    slots = tokens * top
    ex = dbf.Experts(W, count, slots, act=act)
    index = torch.zeros(slots, dtype=torch.int32, device="cuda")
    x = torch.zeros(tokens, m, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros(slots, n, dtype=torch.bfloat16, device="cuda")

    def fill(gen):
        index.copy_(_index(torch, gen, slots, count))
        x.normal_(generator=gen)
        dy.normal_(generator=gen)

    def step():
        g = dbf.group_rows(index, count)
        return ex(x, g, gather=top), ex.backward_data(dy, g, gather=1, scatter=True)

    try:
        _replays(torch, step, fill)
    finally:
        ex.close()


@pytest.mark.parametrize("rows,count,n,m,rank", [(2048, 8, 2056, 2112, 64), (8192, 1, 520, 1032, 16), (2500, 70, 1701, 203, 100)])
def test_adapters(gpu, rows, count, n, m, rank):
    import torch
    print(f"[case] captured adapters {rows} rows of {count}, {n} x {m}, rank {rank}", flush=True)
    gen = torch.Generator(device="cuda").manual_seed(2)
    new = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()  # noqa: E731
    ad = dbf.Adapters(new(count, rank, m), new(count, n, rank))
    index = torch.zeros(rows, dtype=torch.int32, device="cuda")
    x, base, dy = new(rows, m), new(rows, n), new(rows, n)

    def fill(gen):
        index.copy_(_index(torch, gen, rows, count))
        for v in (x, base, dy):
            v.normal_(generator=gen)

    def step():
        g = dbf.group_rows(index, count)
        y, t = ad(x, base, g)
        return (y, t) + ad.backward(dy, x, t, g)

    _replays(torch, step, fill)
