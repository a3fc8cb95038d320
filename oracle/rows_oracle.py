"""fp64 oracle of rows in groups: the grouped order, the products of experts and the low-rank adapters.

Everything is numpy in float64, written from the definitions in
include/dbf.h ("Rows in groups"); nothing is shared with the library.
"""

from __future__ import annotations

import numpy as np


def group_rows(index, count: int):
    """(order, offsets): the rows of each group in rising order, those of no group last."""
    lists = [[] for _ in range(count + 1)]
    for row, v in enumerate(int(i) for i in index):
        lists[v if 0 <= v < count else count].append(row)
    offsets = np.cumsum([0] + [len(part) for part in lists[:count]])
    return np.array([row for part in lists for row in part], dtype=np.int64), offsets.astype(np.int64)


def places(order, offsets):
    """Group of every place of the grouped order (count: none)."""
    count = len(offsets) - 1
    out = np.full(len(order), count)
    for e in range(count):
        out[offsets[e]:offsets[e + 1]] = e
    return out


def experts(x, weights, order, offsets, gather: int, scatter: bool):
    """out[place] = x[row of the place] weights[e].T (weights: a list of 2-D arrays), zeros without a group."""
    out = np.zeros((len(order), weights[0].shape[0]))
    for at, e in enumerate(places(order, offsets)):
        if e < len(weights):
            row = order[at] // gather if gather else at
            out[order[at] if scatter else at] = weights[e] @ x[row]
    return out


def adapters(x, base, A, B, scale, index):
    """(y, t) of low-rank adapters."""
    y, t = np.array(base, np.float64), np.zeros((x.shape[0], A.shape[1]))
    for r, a in enumerate(index):
        if 0 <= a < A.shape[0]:
            t[r] = A[a] @ x[r]
            y[r] += scale[a] * (B[a] @ t[r])
    return y, t


def adapters_backward(dy, x, t, dx, A, B, scale, index):
    """(dx', u, dA, dB)."""
    out, u = np.array(dx, np.float64), np.zeros((x.shape[0], A.shape[1]))
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    for r, a in enumerate(index):
        if 0 <= a < A.shape[0]:
            u[r] = scale[a] * (B[a].T @ dy[r])
            out[r] += A[a].T @ u[r]
            dA[a] += np.outer(u[r], x[r])
            dB[a] += scale[a] * np.outer(dy[r], t[r])
    return out, u, dA, dB
