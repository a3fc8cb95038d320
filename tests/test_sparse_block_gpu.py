"""GPU: rows in groups as a program uses them: a norm, a projection with adapters beside it, a sparse MLP of 4-bit
experts, and the way back, in one captured step; and sizes whose elements pass 32 bits.

Each operator's result is compared with the fp64 oracle at the values that it
was given (so that no tolerance has to hold for a chain), with the tolerances
of the operators' own tests.  Every case prints its name before it touches the
GPU.
"""

import numpy as np
import pytest

import dbf_linear_fwd_amd as dbf
from oracle import mx_oracle as M
from oracle import rows_oracle as O
from tests import test_adapters_gpu as A_
from tests import test_experts_gpu as E_

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _np(t):
    return t.double().cpu().numpy()


def _values(q):
    """fp64 values of an MxTensor."""
    codes, scales = M.unpad_rows(q.codes.cpu().numpy(), q.scales.cpu().numpy(), q.cols, q.fmt)
    return M.values(codes, scales, q.fmt)


class Block:
    """tokens x wide -> norm -> projection + adapters -> up and down projections of two of five experts."""

    def __init__(self, rng, tokens, wide, inner):
        torch = _torch()
        self.tokens, self.wide, self.inner, self.count, self.top, self.requests = tokens, wide, inner, 5, 2, 3
        self.up, self.up_w = E_.make(rng, self.count, inner, wide, tokens * self.top)
        self.down, self.down_w = E_.make(rng, self.count, wide, inner, tokens * self.top)
        codes, s = M.quantize(rng.standard_normal((wide, wide)) * 0.05, "e2m1")
        self.proj_w = M.values(codes, s, "e2m1")
        self.proj = dbf.Layer.mx(E_.blocks_to_dev(codes, s, wide, "e2m1"), max_batch=tokens)
        dev = lambda v: torch.from_numpy(v).to(torch.bfloat16).cuda()  # noqa: E731
        self.ad = dbf.Adapters(dev(rng.standard_normal((self.requests, 8, wide)) / wide ** 0.5),
                               dev(rng.standard_normal((self.requests, wide, 8)) * 0.2),
                               torch.tensor([0.5, 1.0, 2.0], device="cuda"))
        self.weight = dev(1 + 0.1 * rng.standard_normal(wide))
        self.x = torch.zeros(tokens, wide, dtype=torch.bfloat16, device="cuda")
        self.dout = torch.zeros(tokens, wide, dtype=torch.bfloat16, device="cuda")
        self.gates = torch.zeros(tokens, self.top, dtype=torch.float32, device="cuda")
        self.routes = torch.zeros(tokens * self.top, dtype=torch.int32, device="cuda")
        self.request = torch.zeros(tokens, dtype=torch.int32, device="cuda")

    def set(self, rng):
        torch = _torch()
        put = lambda t, v: t.copy_(torch.from_numpy(np.ascontiguousarray(v)).to(t.dtype))  # noqa: E731
        put(self.x, rng.standard_normal((self.tokens, self.wide)))
        put(self.dout, rng.standard_normal((self.tokens, self.wide)) * 0.01)
        put(self.gates, rng.random((self.tokens, self.top)))
        ids = np.argsort(rng.random((self.tokens, self.count)), axis=1)[:, :self.top]
        ids[-3:] = -1  # a padded batch
        put(self.routes, ids.reshape(-1))
        put(self.request, np.where(rng.random(self.tokens) < 0.2, -1, rng.integers(0, self.requests, self.tokens)))

    def step(self):
        torch = _torch()
        r = {}
        groups = dbf.group_rows(self.routes, self.count)
        mine = dbf.group_rows(self.request, self.requests)
        r["norm"] = dbf.rms_norm(self.x, self.weight)
        r["base"] = self.proj(r["norm"].y)
        r["h"], r["t"] = self.ad(r["norm"].y, r["base"], mine)
        r["q"] = dbf.mx_quantize(r["h"], "e4m3")
        r["a"] = self.up(r["q"], groups, gather=self.top, out_dtype=torch.bfloat16)
        r["b"] = torch.relu(r["a"])
        r["c"] = self.down(r["b"], groups, scatter=True)
        gates = self.gates.to(torch.bfloat16)
        r["y"] = (r["c"].view(self.tokens, self.top, self.wide) * gates[:, :, None]).sum(1)
        # back
        r["dc"] = (self.dout[:, None, :] * gates[:, :, None]).reshape(-1, self.wide).contiguous()
        r["db"] = self.down.backward_data(r["dc"], groups, gather=1)
        r["da"] = torch.where(r["a"] > 0, r["db"], torch.zeros_like(r["db"]))
        r["dslots"] = self.up.backward_data(r["da"], groups, scatter=True)
        r["dh"] = r["dslots"].view(self.tokens, self.top, self.wide).sum(1)
        r["dbase"] = self.proj.backward_data(r["dh"])
        r["dn"], r["dA"], r["dB"] = self.ad.backward(r["dh"], r["norm"].y, r["t"], mine, dx=r["dbase"])
        r["dx"], r["dw"] = dbf.rms_norm_backward(r["dn"], r["norm"].h, self.weight, r["norm"].rstd)
        return r

    def check(self, r):
        torch = _torch()
        order, offsets = O.group_rows(self.routes.cpu().numpy(), self.count)
        place = O.places(order, offsets)

        def product(got, xv, w, K, gather, scatter, e4m3):
            ref = O.experts(xv, w, order, offsets, gather, scatter)
            mag = O.experts(np.abs(xv), [np.abs(v) for v in w], order, offsets, gather, scatter)
            lost = np.zeros_like(ref)
            if e4m3:
                for at, e in enumerate(place):
                    if e < self.count:
                        row = order[at] // gather if gather else at
                        lost[order[at] if scatter else at] = 7 * 2.0 ** -13 * E_.cut(xv[row][None], w[e])[0]
            E_.check(got, ref, mag, K, "bf16", lost)

        product(r["a"], _values(r["q"]), self.up_w, self.wide, self.top, False, True)
        product(r["c"], M.values(*M.quantize(_np(r["b"]), "e4m3"), "e4m3"), self.down_w, self.inner, 0, True, True)
        product(r["db"], _np(r["dc"]), [w.T for w in self.down_w], self.wide, 1, False, False)
        product(r["dslots"], _np(r["da"]), [w.T for w in self.up_w], self.inner, 0, True, False)
        index = self.request.cpu().numpy()
        half, m = torch.finfo(torch.bfloat16).eps / 2, self.wide
        A, B, s, x = _np(self.ad.A), _np(self.ad.B), _np(self.ad.scale), _np(r["norm"].y)
        y, t = O.adapters(x, _np(r["base"]), A, B, s, index)
        _, tm = O.adapters(np.abs(x), np.abs(_np(r["base"])), np.abs(A), np.abs(B), s, index)
        te = (m / 8 + 16) * 2.0 ** -24 * tm
        A_.within(_np(r["t"]), t, te, "t")
        loose = te + 2.0 ** -17 * (np.abs(t) + te) + 20 * 2.0 ** -24 * (np.abs(t) + te)
        ye = 2.0 ** -24 * np.abs(y)
        for row, a in enumerate(index):
            if a >= 0:
                ye[row] += s[a] * (np.abs(B[a]) @ loose[row])
        A_.within(_np(r["h"]), y, ye + half * (np.abs(y) + ye), "adapters")
        none = torch.from_numpy(np.flatnonzero(self.routes.cpu().numpy() < 0)).cuda()
        assert not bool(r["c"][none].any()) and not bool(r["dslots"][none].any())
        for v in r.values():
            if isinstance(v, torch.Tensor):
                assert bool(torch.isfinite(v.float()).all())


@pytest.mark.parametrize("tokens,wide,inner", [(1 + 3, 256, 384), (37, 320, 200), (300, 256, 512)])
def test_block_eager_and_captured(gpu, tokens, wide, inner):
    E_._say(f"block {tokens} tokens {wide} {inner}")
    torch = _torch()
    block = Block(np.random.default_rng(tokens), tokens, wide, inner)
    block.set(np.random.default_rng(1))
    block.check(block.step())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block.step()
    for seed in (2, 3, 4):
        block.set(np.random.default_rng(seed))
        graph.replay()
        got = {k: v.clone() for k, v in held.items() if isinstance(v, torch.Tensor)}
        torch.cuda.synchronize()
        want = block.step()
        for k, v in got.items():
            # (torch's own sum over two slots is elementwise: equal as well)
            assert torch.equal(v, want[k]), k
    block.check(block.step())


def test_two_streams_with_handles_of_their_own(gpu):
    """Experts on two streams at once, each with its handle, adapters from one object on both."""
    torch = _torch()
    rng = np.random.default_rng(17)
    count, n, m, slots = 4, 256, 512, 600
    pair = [E_.make(np.random.default_rng(3), count, n, m, slots)[0] for _ in range(2)]
    g, _ = E_.group(rng.integers(0, count, slots), count)
    ad = dbf.Adapters(torch.randn(count, 16, m, device="cuda").half(), torch.randn(count, n, 16, device="cuda").half())
    xs = [torch.randn(slots, m, device="cuda").half() for _ in range(2)]
    base = torch.randn(slots, n, device="cuda").half()
    want = [(ex(x, g), ad(x, base, g).y) for ex, x in zip(pair, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for turn in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append((pair[i](xs[i], g), ad(xs[i], base, g).y))
    torch.cuda.synchronize()
    for i in range(2):
        for y, z in got[i]:
            assert torch.equal(y, want[i][0]) and torch.equal(z, want[i][1])


def test_adapters_past_32_bits(gpu):
    """More than 2^31 elements in the layer's results: the last rows and columns."""
    E_._say("adapters 70000 x 32768")
    torch = _torch()
    rows, n, m, rank = 70000, 32768, 64, 4
    gen = torch.Generator(device="cuda").manual_seed(1)
    index = torch.randint(-1, 3, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    index[-1] = 2
    g = dbf.group_rows(index, 3)
    A = torch.randn(3, rank, m, generator=gen, device="cuda").bfloat16()
    B = torch.randn(3, n, rank, generator=gen, device="cuda").bfloat16()
    x = torch.randn(rows, m, generator=gen, device="cuda").bfloat16()
    base = torch.randn(rows, n, generator=gen, device="cuda", dtype=torch.bfloat16)
    ad = dbf.Adapters(A, B)
    y, t = ad(x, base, g)
    for at in (slice(0, 40), slice(rows - 40, rows)):
        ids = index[at].long()
        on = (ids >= 0)[:, None]
        low = torch.where(on, torch.einsum("rm,rkm->rk", x[at].double(), A[ids].double()), 0.0)
        ref = base[at].double() + torch.einsum("rk,rnk->rn", low, B[ids].double())
        # half a step, and what the sums and t's parts may add: 2^-16 of Σ|B||t|
        mag = torch.einsum("rk,rnk->rn", low.abs(), B[ids].double().abs())
        assert bool(((y[at].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -15 * mag + 1e-30).all())
    dx, dA, dB = ad.backward(base, x, t, g)
    cols = slice(n - 64, n)
    for a in range(3):
        on = index == a
        ref = base[on][:, cols].double().t() @ t[on].double()
        mag = base[on][:, cols].double().abs().t() @ t[on].double().abs()
        assert bool(((dB[a, cols].double() - ref).abs() <= (3 * rows / 8 + 40) * 2.0 ** -24 * mag).all())
    last = (base[-1].double() @ B[2].double()) @ A[2].double()
    mag = (base[-1].double().abs() @ B[2].double().abs()) @ A[2].double().abs()
    assert bool(((dx[-1].double() - last).abs() <= 2.0 ** -8 * last.abs() + (n / 8 + 600) * 2.0 ** -24 * mag).all())


def test_expert_weights_past_32_bits(gpu):
    """Weights of more than 2^32 bytes: the first and the last expert, bit for bit as layers of their own (whole and
    half numbers: every sum is exact)."""
    E_._say("experts 44 x 14336 x 14336")
    torch = _torch()
    count, n, m = 44, 14336, 14336
    codes = torch.randint(0, 256, (count * n, m // 2), device="cuda", dtype=torch.uint8)
    scales = torch.full((count * n, m // 32), 127, device="cuda", dtype=torch.uint8)
    assert codes.numel() > 2 ** 32
    ex = dbf.Experts(dbf.MxTensor(codes, scales, m, "e2m1"), count, max_rows=40)
    index = torch.tensor([0, count - 1, -1] * 13, dtype=torch.int32, device="cuda")
    x = torch.randint(-1, 2, (39, m), device="cuda").half()
    dy = torch.randint(-1, 2, (39, n), device="cuda").half()
    g = dbf.group_rows(index, count)
    y = ex(x, g, gather=1, scatter=True)
    dx = ex.backward_data(dy, g, gather=1, scatter=True)
    for e in (0, count - 1):
        at = slice(e * n, (e + 1) * n)
        layer = dbf.Layer.mx(dbf.MxTensor(codes[at].contiguous(), scales[at].contiguous(), m, "e2m1"), max_batch=13)
        mine = index == e
        assert torch.equal(y[mine], layer(x[mine].contiguous()))
        assert torch.equal(dx[mine], layer.backward_data(dy[mine].contiguous()))
        layer.close()
    assert not bool(y[index < 0].any()) and not bool(dx[index < 0].any())
    ex.close()
