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

The calls write into tensors, like the LoRA calls, and automatic differentiation does not see
them: a training program calls the two gradients itself, or wraps the three products in a
``torch.autograd.Function``.  Work given to a ``stream`` is ordered on that stream alone.
"""
from __future__ import annotations

import contextlib
import dataclasses
from typing import Optional

from . import _lib
from ._lib import check, check_sizes
from .sgmv import _check_rows, _torch, dtype_code


def _on(stream):
    """Allocations made for work on ``stream`` belong to it."""
    return contextlib.nullcontext() if stream is None else _torch().cuda.stream(stream)


def _stream_of(stream, *tensors) -> int:
    """The handle of ``stream`` (None: the current one), once every tensor is known to be on the
    current GPU, where the kernels are launched.  (The raw handle is taken directly: building a
    Stream object costs as much as the launch.)"""
    torch = _torch()
    here = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != here:
            raise ValueError("tensors must be on one GPU")
    if here < 0 or here != torch.cuda.current_device():
        raise ValueError("tensors must be on the current GPU")
    return torch._C._cuda_getCurrentRawStream(here) if stream is None else int(stream.cuda_stream)


@dataclasses.dataclass
class RowGroups:
    """Group tables on the device (see sgmv_group_rows), int32 [n_groups + 1 + n]: rows
    ``perm[starts[g]:starts[g + 1]]`` belong to group g, rows ``perm[starts[n_groups]:]`` to
    none."""
    n: int
    n_groups: int
    table: object

    @property
    def starts(self):
        return self.table[: self.n_groups + 1]

    @property
    def perm(self):
        return self.table[self.n_groups + 1:]


def group_rows(ids, n_groups: int, stream=None) -> RowGroups:
    """Group tables of a batch whose row i has the id ``ids[i]`` (device int32 [n])."""
    if ids.dtype != _torch().int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a device int32 tensor [n]")
    handle = _stream_of(stream, ids)
    n = ids.shape[0]
    check_sizes("sgmv_group_rows", n)
    if not 1 <= n_groups <= _lib.MAX_GROUPS:
        check(_lib.ERR_SHAPE if n_groups < 1 else _lib.ERR_UNSUPPORTED, "sgmv_group_rows")
    if stream is None:
        table = ids.new_empty(n + n_groups + 1)
    else:
        with _on(stream):
            table = ids.new_empty(n + n_groups + 1)
    at = table.data_ptr()
    st = _lib.lib().sgmv_group_rows(handle, ids.data_ptr(), n, n_groups, at + 4 * (n_groups + 1), at)
    check(st, "sgmv_group_rows")
    return RowGroups(n, n_groups, table)


def _tables(groups: Optional[RowGroups], n: int, like):
    """(starts, perm, n_groups) for the C calls; None makes all rows one group."""
    if groups is None:
        return None, None, 1
    if groups.n != n:
        raise ValueError(f"{n} rows, but the groups were made of {groups.n}")
    table, E = groups.table, groups.n_groups
    if table.dtype is not _torch().int32 or table.shape != (E + 1 + n,) or not table.is_contiguous():
        raise ValueError(f"groups must hold a dense int32 table [{E + 1 + n}], as group_rows makes it")
    if table.get_device() != like.get_device():
        raise ValueError("groups must be on the tensors' GPU")
    at = table.data_ptr()
    return at, at + 4 * (E + 1), E


def _share(n: int, x_rows: int) -> int:
    if x_rows == 0 or n % x_rows != 0:
        if n == 0:
            return 1
        raise ValueError(f"{n} rows cannot share the {x_rows} rows of x evenly")
    return max(n // x_rows, 1)


def _ld(t) -> int:
    """Elements between the rows of a matrix; one row may have any stride."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


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


def _same_type(a, b, c):
    if b.dtype != a.dtype or c.dtype != a.dtype:
        raise TypeError("all operands must share a dtype")
    return dtype_code(a)


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
    check_sizes("sgmv_group_matmul", n, h_in, h_out)
    dt, share = _same_type(y, x, W), _share(n, int(x.shape[0]))
    starts, perm, E = _tables(groups, n, y)
    handle = _stream_of(stream, y, x, W)
    st = _lib.lib().sgmv_group_matmul(handle, dt, y.data_ptr(), _ld(y),
                                      x.data_ptr(), _ld(x), share, W.data_ptr(), stride,
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
    check_sizes("sgmv_group_matmul_dx", n, h_in, h_out)
    dt = _same_type(dx, dy, W)
    starts, perm, E = _tables(groups, n, dx)
    handle = _stream_of(stream, dx, dy, W)
    st = _lib.lib().sgmv_group_matmul_dx(handle, dt, dx.data_ptr(), _ld(dx),
                                         dy.data_ptr(), _ld(dy), W.data_ptr(), stride,
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
    check_sizes("sgmv_group_matmul_dw", n, h_in, h_out)
    dt, share = _same_type(dW, x, dy), _share(n, int(x.shape[0]))
    starts, perm, E = _tables(groups, n, dW)
    handle = _stream_of(stream, dW, x, dy)
    st = _lib.lib().sgmv_group_matmul_dw(handle, dt, dW.data_ptr(), stride,
                                         x.data_ptr(), _ld(x), share, dy.data_ptr(),
                                         _ld(dy), starts, perm, n, E, h_in, h_out)
    check(st, "sgmv_group_matmul_dw")
    return dW
