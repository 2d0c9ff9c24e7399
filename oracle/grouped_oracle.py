"""Plain fp64 definitions of the products grouped by row ids and of the microscaled 4-bit
format (MX), on numpy arrays.  Shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

MX_BLOCK = 32
MX_VALUES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# --------------------------------------------------------------------------------------
# rows grouped by id
# --------------------------------------------------------------------------------------
def group_rows(ids, n_groups: int):
    """(starts int32 [G + 1], perm int32 [n]): rows in order of (group, row), rows whose id
    lies outside [0, G) last."""
    ids = np.asarray(ids, np.int64)
    key = np.where((ids >= 0) & (ids < n_groups), ids, n_groups)
    perm = np.argsort(key, kind="stable").astype(np.int32)
    starts = np.searchsorted(key[perm], np.arange(n_groups + 1)).astype(np.int32)
    return starts, perm


def _of_group(ids, g):
    return np.flatnonzero(np.asarray(ids) == g)


def group_matmul(x, W, ids, share: int = 1):
    """(y, m): y[i] = x[i // share] @ W[ids[i]].T and m, the same of the magnitudes (what
    rounding errors of the sum are measured by); rows of no group are zero."""
    n = len(ids)
    y = np.zeros((n, W.shape[1]))
    m = np.zeros_like(y)
    for g in range(W.shape[0]):
        rows = _of_group(ids, g)
        if len(rows):
            y[rows] = x[rows // share] @ W[g].T
            m[rows] = np.abs(x[rows // share]) @ np.abs(W[g]).T
    return y, m


def group_matmul_dx(dy, W, ids):
    """(dx, m): dx[i] = dy[i] @ W[ids[i]]."""
    dx = np.zeros((len(ids), W.shape[2]))
    m = np.zeros_like(dx)
    for g in range(W.shape[0]):
        rows = _of_group(ids, g)
        if len(rows):
            dx[rows] = dy[rows] @ W[g]
            m[rows] = np.abs(dy[rows]) @ np.abs(W[g])
    return dx, m


def group_matmul_dw(x, dy, ids, n_groups: int, share: int = 1):
    """(dW, m): dW[g] = sum over the rows i of group g of dy[i].T x[i // share]."""
    dW = np.zeros((n_groups, dy.shape[1], x.shape[1]))
    m = np.zeros_like(dW)
    for g in range(n_groups):
        rows = _of_group(ids, g)
        if len(rows):
            dW[g] = dy[rows].T @ x[rows // share]
            m[g] = np.abs(dy[rows]).T @ np.abs(x[rows // share])
    return dW, m


# --------------------------------------------------------------------------------------
# MX
# --------------------------------------------------------------------------------------
def mx_encode(v):
    """(codes uint8 [.., h / 2], scales uint8 [.., h / 32]) of float64 values v [.., h]."""
    b = np.asarray(v, np.float64).reshape(*v.shape[:-1], -1, MX_BLOCK)
    finite = np.isfinite(b).all(-1)
    b = np.where(finite[..., None], b, 0.0)
    top = np.abs(b).max(-1)
    e = np.where(top > 0, np.frexp(np.where(top > 0, top, 1.0))[1] - 1 - 2, -127)
    e = np.maximum(e, -127)
    a = np.abs(b) / np.exp2(e)[..., None]
    # nearest of the eight values, the even code where two are equally near
    d = np.abs(a[..., None] - MX_VALUES)
    best = d.min(-1, keepdims=True)
    near = d == best
    code = np.argmax(near, -1)
    tie = near.sum(-1) == 2
    code = np.where(tie & (code % 2 == 1), code + 1, code)
    code = np.where(np.signbit(b) & finite[..., None], code + 8, code).reshape(v.shape)
    scales = np.where(finite, e + 127, 255).astype(np.uint8)
    return (code[..., 0::2] + 16 * code[..., 1::2]).astype(np.uint8), scales


def mx_decode(codes, scales):
    """float64 values of codes and scales; scale byte 255 is NaN."""
    c = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], -1)
    v = np.where(c >= 8, -MX_VALUES[c & 7], MX_VALUES[c & 7])
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return v * np.repeat(s, MX_BLOCK, -1)
