"""Products grouped by row ids (expert layers) and their gradients, on torch tensors.

Argument checks and marshalling only: every step runs in libsgmv's HIP kernels
(``sgmv_group_*`` in include/sgmv.h).  A layer of E experts holds ``W [E, h_out, h_in]``;
its router gives every row an id in [0, E), or one outside that range for a row that is not
computed here::

    groups = group_rows(ids, E)                  # once per batch and layer, on the device
    group_matmul(y, x, W, groups)                # y[i] = x[i // share] @ W[ids[i]].T
    group_matmul_dx(dx, dy, W, groups)           # dx[i] = dy[i] @ W[ids[i]]
    group_matmul_dw(dW, x, dy, groups)           # dW[e] = sum of dy[i].T x[i // share]

``share`` is how many consecutive rows read one row of x (the experts per token): the rows
of the other operand over the rows of x.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

from . import _lib
from ._lib import check
from .sgmv import _check_rows, _stream_handle, _torch, dtype_code


def _on(stream):
    """Allocations made for work on ``stream`` belong to it."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _check_device(*tensors):
    """Every tensor is on the current GPU (the kernels are launched there)."""
    here = _torch().cuda.current_device() if tensors[0].is_cuda else -1
    for t in tensors:
        if t.get_device() != here or here < 0:
            raise ValueError("tensors must be on the current GPU")


@dataclasses.dataclass
class RowGroups:
    """Group tables on the device (see sgmv_group_rows): rows ``perm[starts[g]:starts[g + 1]]``
    belong to group g, rows ``perm[starts[n_groups]:]`` to none."""
    n: int
    n_groups: int
    starts: object   # int32 [n_groups + 1]
    perm: object     # int32 [n]


def group_rows(ids, n_groups: int, stream=None) -> RowGroups:
    """Group tables of a batch whose row i has the id ``ids[i]`` (device int32 [n])."""
    torch = _torch()
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a device int32 tensor [n]")
    _check_device(ids)
    n = int(ids.shape[0])
    with _on(stream):
        table = torch.empty(n + n_groups + 1, dtype=torch.int32, device=ids.device)
    starts, perm = table[: n_groups + 1], table[n_groups + 1:]
    st = _lib.lib().sgmv_group_rows(_stream_handle(stream), ids.data_ptr(), n, n_groups,
                                    perm.data_ptr(), starts.data_ptr())
    check(st, "sgmv_group_rows")
    return RowGroups(n, n_groups, starts, perm)


def _tables(groups: Optional[RowGroups], n: int):
    """(starts, perm, n_groups) for the C calls; None makes all rows one group."""
    if groups is None:
        return None, None, 1
    if groups.n != n:
        raise ValueError(f"{n} rows, but the groups were made of {groups.n}")
    _check_device(groups.starts, groups.perm)
    return groups.starts.data_ptr(), groups.perm.data_ptr(), groups.n_groups


def _share(n: int, x_rows: int) -> int:
    if x_rows == 0 or n % x_rows != 0:
        if n == 0:
            return 1
        raise ValueError(f"{n} rows cannot share the {x_rows} rows of x evenly")
    return max(n // x_rows, 1)


def _pool(W, groups: Optional[RowGroups], name: str):
    """A weight [E, h_out, h_in] (or [h_out, h_in] without groups): (h_out, h_in, stride)."""
    E = 1 if groups is None else groups.n_groups
    if W.dim() == 2 and groups is None:
        W = W.unsqueeze(0)
    if W.dim() != 3 or W.shape[0] != E:
        raise ValueError(f"{name} must be [{E}, h_out, h_in]")
    h_out, h_in = int(W.shape[1]), int(W.shape[2])
    if W.stride(2) != 1 or W.stride(1) != h_in:
        raise ValueError(f"{name} must hold dense row-major groups")
    return h_out, h_in, (W.stride(0) if E > 1 else h_out * h_in)


def _same_type(*tensors):
    if any(t.dtype != tensors[0].dtype for t in tensors):
        raise TypeError("all operands must share a dtype")
    return dtype_code(tensors[0])


def group_matmul(y, x, W, groups: Optional[RowGroups] = None, stream=None):
    """y[i] = x[i // share] @ W[g].T for the rows i of every group g; rows of no group get
    zeros.  ``groups=None`` is the dense product with one W."""
    n = int(y.shape[0])
    _check_rows(y, n, "y")
    _check_rows(x, x.shape[0], "x")
    h_out, h_in, stride = _pool(W, groups, "W")
    if x.shape[1] != h_in or y.shape[1] != h_out:
        raise ValueError(f"x [., {x.shape[1]}] / y [., {y.shape[1]}] do not match W's "
                         f"h_in = {h_in}, h_out = {h_out}")
    dt, share = _same_type(y, x, W), _share(n, int(x.shape[0]))
    starts, perm, E = _tables(groups, n)
    _check_device(y, x, W)
    st = _lib.lib().sgmv_group_matmul(_stream_handle(stream), dt, y.data_ptr(), y.stride(0),
                                      x.data_ptr(), x.stride(0), share, W.data_ptr(), stride,
                                      starts, perm, n, E, h_in, h_out)
    check(st, "sgmv_group_matmul")
    return y


def group_matmul_dx(dx, dy, W, groups: Optional[RowGroups] = None, stream=None):
    """dx[i] = dy[i] @ W[g] for the rows i of every group g; rows of no group get zeros.
    Where rows share an x, its gradient is the sum of theirs."""
    n = int(dy.shape[0])
    _check_rows(dy, n, "dy")
    _check_rows(dx, n, "dx")
    h_out, h_in, stride = _pool(W, groups, "W")
    if dx.shape[1] != h_in or dy.shape[1] != h_out:
        raise ValueError(f"dx [., {dx.shape[1]}] / dy [., {dy.shape[1]}] do not match W's "
                         f"h_in = {h_in}, h_out = {h_out}")
    dt = _same_type(dx, dy, W)
    starts, perm, E = _tables(groups, n)
    _check_device(dx, dy, W)
    st = _lib.lib().sgmv_group_matmul_dx(_stream_handle(stream), dt, dx.data_ptr(), dx.stride(0),
                                         dy.data_ptr(), dy.stride(0), W.data_ptr(), stride,
                                         starts, perm, n, E, h_in, h_out)
    check(st, "sgmv_group_matmul_dx")
    return dx


def group_matmul_dw(dW, x, dy, groups: Optional[RowGroups] = None, stream=None):
    """dW[g] = sum over the rows i of group g of dy[i].T x[i // share], overwritten (zeros for
    a group without rows)."""
    n = int(dy.shape[0])
    _check_rows(dy, n, "dy")
    _check_rows(x, x.shape[0], "x")
    h_out, h_in, stride = _pool(dW, groups, "dW")
    if x.shape[1] != h_in or dy.shape[1] != h_out:
        raise ValueError(f"x [., {x.shape[1]}] / dy [., {dy.shape[1]}] do not match dW's "
                         f"h_in = {h_in}, h_out = {h_out}")
    dt, share = _same_type(dW, x, dy), _share(n, int(x.shape[0]))
    starts, perm, E = _tables(groups, n)
    _check_device(dW, x, dy)
    st = _lib.lib().sgmv_group_matmul_dw(_stream_handle(stream), dt, dW.data_ptr(), stride,
                                         x.data_ptr(), x.stride(0), share, dy.data_ptr(),
                                         dy.stride(0), starts, perm, n, E, h_in, h_out)
    check(st, "sgmv_group_matmul_dw")
    return dW
