"""Pins of the block-format and norm oracle (CPU)."""

import numpy as np
import pytest

from oracle import mx_oracle as O


def test_code_tables():
    e2 = O.code_values("e2m1")
    assert list(e2[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert list(e2[8:]) == [-0.0, -0.5, -1, -1.5, -2, -3, -4, -6]
    e4 = O.code_values("e4m3")
    assert e4[0x7e] == 448 and e4[0x01] == 2.0 ** -9 and e4[0x08] == 2.0 ** -6 and e4[0x38] == 1.0
    assert np.isnan(e4[0x7f]) and np.isnan(e4[0xff])
    assert np.all(np.diff(e4[:0x7f]) > 0)


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_nearest_code_by_exhaustive_distance(fmt):
    """Nearest by comparing with every value; every midpoint goes to the even code."""
    half = 128 if fmt == "e4m3" else 8
    pos = O.code_values(fmt)[:half]
    n = int(np.isfinite(pos).sum())
    pos = pos[:n]
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(0, pos[-1] * 1.2, 4000), np.exp2(rng.uniform(-12, 9, 4000)), pos,
                        (pos[1:] + pos[:-1]) / 2])
    got = O.nearest_code(v, fmt)
    d = np.abs(v[:, None] - pos[None, :])
    best = d.min(axis=1)
    for i, c in enumerate(got):
        cand = np.nonzero(d[i] == best[i])[0]
        assert c in cand
        if len(cand) > 1:
            assert c % 2 == 0
    assert np.array_equal(O.nearest_code(-v, fmt), got + half)


def test_quantize_worked_example():
    x = np.zeros((1, 40))
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 7.0, -2.5, 0.25, 0.75
    x[0, 39] = 2.0 ** -130  # second block: the scale byte clamps at 0
    codes, s = O.quantize(x, "e2m1")
    # amax 7: floor(log2 7) - 2 = 0, so byte 127; 7 saturates at 6, 2.5 ties to 2, 0.25 ties to 0, 0.75 to 1
    assert s[0, 0] == 127
    assert list(codes[0, :4]) == [7, 8 + 4, 0, 2]
    assert s[0, 1] == 0 and codes[0, 39] == O.nearest_code(np.array([2.0 ** -3]), "e2m1")[0]
    x[0, 5] = np.inf
    codes, s = O.quantize(x, "e2m1")
    assert s[0, 0] == 255 and not codes[0, :32].any() and s[0, 1] == 0
    assert np.isnan(O.values(codes, s, "e2m1")[0, :32]).all()


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
def test_layout_round_trip(fmt):
    rng = np.random.default_rng(1)
    codes, s = O.quantize(rng.standard_normal((5, 300)), fmt)
    c, sc = O.pad_rows(codes, s, fmt)
    assert c.shape == (5, 384 if fmt == "e4m3" else 192) and sc.shape == (5, 12)
    c2, s2 = O.unpad_rows(c, sc, 300, fmt)
    assert np.array_equal(c2, codes) and np.array_equal(s2, s)


def test_norm_gradient_against_differences():
    rng = np.random.default_rng(2)
    h, w, dy = rng.standard_normal((3, 17)), rng.standard_normal(17), rng.standard_normal((3, 17))
    eps = 1e-3
    _, rstd = O.rms_norm(h, w, eps)
    dx, dw = O.rms_norm_backward(dy, h, w, rstd)
    f = lambda hh, ww: float((O.rms_norm(hh, ww, eps)[0] * dy).sum())  # noqa: E731
    d = 1e-6
    for r in range(3):
        for c in range(17):
            e = np.zeros_like(h)
            e[r, c] = d
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * d) - dx[r, c]) < 1e-7
    for c in range(17):
        e = np.zeros_like(w)
        e[c] = d
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * d) - dw[c]) < 1e-7


def test_linear_gradient_against_differences():
    rng = np.random.default_rng(3)
    w, x, dy = rng.standard_normal((7, 11)), rng.standard_normal((2, 11)), rng.standard_normal((2, 7))
    dx, _ = O.backward_data(dy, w)
    for r in range(2):
        for c in range(11):
            e = np.zeros_like(x)
            e[r, c] = 1.0  # linear in x: any step is exact up to rounding
            assert abs(((O.linear(x + e, w)[0] - O.linear(x, w)[0]) * dy).sum() - dx[r, c]) < 1e-12
