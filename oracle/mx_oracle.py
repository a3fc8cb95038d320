"""fp64 oracle of the block formats, the layers with a 4-bit block weight and the root-mean-square norm.

Everything is numpy in float64, written from the definitions in
include/dbf.h ("Block formats", dbf_mx_forward, dbf_rms_norm); nothing is
shared with the library.
"""

from __future__ import annotations

import numpy as np

# format: exponent of the largest value
EMAX = {"e4m3": 8, "e2m1": 2}


def code_values(fmt: str) -> np.ndarray:
    """Value of every code (256 for e4m3, 16 for e2m1), from sign, exponent and mantissa fields."""
    bits, ebits, mbits, bias = (8, 4, 3, 7) if fmt == "e4m3" else (4, 2, 1, 1)
    out = np.empty(1 << bits)
    for c in range(1 << bits):
        man = c & ((1 << mbits) - 1)
        ex = (c >> mbits) & ((1 << ebits) - 1)
        if fmt == "e4m3" and ex == 15 and man == 7:
            v = np.nan
        elif ex == 0:
            v = man * 2.0 ** (1 - bias - mbits)
        else:
            v = (1 + man / (1 << mbits)) * 2.0 ** (ex - bias)
        out[c] = -v if c >> (bits - 1) else v
    return out


def nearest_code(v: np.ndarray, fmt: str) -> np.ndarray:
    """Code of the value nearest to v (ties to the even code, saturating); the sign of a zero is kept."""
    half = 128 if fmt == "e4m3" else 8
    pos = code_values(fmt)[:half]
    pos = pos[np.isfinite(pos)]
    a = np.abs(v)
    hi = np.clip(np.searchsorted(pos, a), 1, len(pos) - 1)  # pos[hi - 1] < a <= pos[hi], or the ends
    lo = hi - 1
    dl, dh = a - pos[lo], pos[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    c = np.where(up, hi, lo)
    return np.where(np.signbit(v), c + half, c)


def quantize(x: np.ndarray, fmt: str):
    """(codes, scale bytes) of x (rows x cols): codes (rows, cols) and scales (rows, ceil(cols / 32))."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    nb = -(-cols // 32)
    full = np.zeros((rows, nb * 32))
    full[:, :cols] = x
    b = full.reshape(rows, nb, 32)
    bad = ~np.isfinite(b).all(axis=2)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=2))
    _, e = np.frexp(amax)  # amax = f 2^e with f in [1/2, 1)
    s = np.where(amax > 0, np.clip(e - 1 - EMAX[fmt] + 127, 0, 254), 0)
    scaled = np.where(bad[:, :, None], 0.0, b * np.exp2(127.0 - s)[:, :, None])
    codes = nearest_code(scaled, fmt)
    codes = np.where(bad[:, :, None], 0, codes)
    s = np.where(bad, 255, s)
    return codes.reshape(rows, nb * 32)[:, :cols].astype(np.uint8), s.astype(np.uint8)


def values(codes: np.ndarray, scales: np.ndarray, fmt: str) -> np.ndarray:
    """fp64 values of codes (rows, cols) and scales (rows, blocks)."""
    sv = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return code_values(fmt)[codes] * np.repeat(sv, 32, axis=1)[:, :codes.shape[1]]


def pad_rows(codes: np.ndarray, scales: np.ndarray, fmt: str):
    """The padded row layout: codes (rows, row bytes) and scales (rows, padded blocks), uint8."""
    rows, cols = codes.shape
    wide = -(-cols // 128) * 128
    c = np.zeros((rows, wide), np.uint8)
    c[:, :cols] = codes
    s = np.zeros((rows, wide // 32), np.uint8)
    s[:, :scales.shape[1]] = scales
    if fmt == "e2m1":
        c = c[:, 0::2] | (c[:, 1::2] << 4)
    return np.ascontiguousarray(c), s


def unpad_rows(codes: np.ndarray, scales: np.ndarray, cols: int, fmt: str):
    """Codes (rows, cols) and scales (rows, blocks) of the padded row layout."""
    if fmt == "e2m1":
        c = np.empty((codes.shape[0], codes.shape[1] * 2), np.uint8)
        c[:, 0::2] = codes & 15
        c[:, 1::2] = codes >> 4
        codes = c
    return codes[:, :cols], scales[:, :-(-cols // 32)]


def linear(xv: np.ndarray, wv: np.ndarray):
    """(y, the sum of the products' magnitudes) for values xv (batch x m) and wv (n x m)."""
    return xv @ wv.T, np.abs(xv) @ np.abs(wv).T


def backward_data(dy: np.ndarray, wv: np.ndarray):
    """(dx, the sum of the products' magnitudes)."""
    dy = np.asarray(dy, np.float64)
    return dy @ wv, np.abs(dy) @ np.abs(wv)


def rms_norm(h: np.ndarray, w: np.ndarray, eps: float):
    """(y, rstd) of rows h."""
    h = np.asarray(h, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h * rstd[:, None] * w[None, :], rstd


def rms_norm_backward(dy: np.ndarray, h: np.ndarray, w: np.ndarray, rstd: np.ndarray):
    """(dx, dweight) of rms_norm at h for the upstream gradient dy."""
    dy = np.asarray(dy, np.float64)
    xh = np.asarray(h, np.float64) * rstd[:, None]
    g = dy * w[None, :]
    dx = rstd[:, None] * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0)
