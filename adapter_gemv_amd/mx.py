"""Microscaled 4-bit floating point (MX) on torch tensors: quantisation, and products with
weights held in it.  Argument checks and marshalling only (``sgmv_mx_*`` in include/sgmv.h,
which defines the format)::

    Wq = mx_quantize(W)                     # W [.., h_out, h_in] once, when it is loaded
    mx_matmul(y, x, Wq, groups)             # y[i] = x[i // share] @ Wq[g].T, x in 16 bits
    mx_matmul(y, mx_quantize(x), Wq, groups)     # both sides in 4 bits
    mx_dequantize(W, Wq)                    # the values back, in W's type
"""
from __future__ import annotations

import dataclasses
from typing import Optional

from . import _lib
from ._lib import check, check_sizes
from .grouped import RowGroups, _ld, _on, _share, _stream_of, _tables
from .sgmv import _check_rows, _torch, dtype_code

BLOCK = 32


@dataclasses.dataclass
class MxTensor:
    """``codes`` uint8 [.., h / 2] (the element at an even place in the low half of its byte)
    and ``scales`` uint8 [.., h / 32] (2^(scale - 127) of each block of 32), both dense."""
    codes: object
    scales: object

    def __post_init__(self):
        uint8 = _torch().uint8
        c, s = self.codes, self.scales
        if c.dtype != uint8 or s.dtype != uint8:
            raise TypeError("codes and scales must be uint8")
        cs, ss = tuple(c.shape), tuple(s.shape)
        if not cs or not ss or cs[:-1] != ss[:-1] or cs[-1] != ss[-1] * (BLOCK // 2):
            raise ValueError(f"codes {tuple(c.shape)} and scales {tuple(s.shape)} do not match: "
                             "[.., h / 2] and [.., h / 32]")
        if not c.is_contiguous() or not s.is_contiguous():
            raise ValueError("codes and scales must be dense")

    @property
    def shape(self):
        """The shape of the values."""
        return (*self.codes.shape[:-1], 2 * self.codes.shape[-1])


def _as_rows(t, name: str):
    """(rows, h, row stride) of a tensor [.., h] whose rows are a fixed distance apart."""
    if t.dim() < 1 or t.shape[-1] == 0 or t.stride(-1) != 1:
        raise ValueError(f"{name} must be [.., h] with unit column stride")
    h = int(t.shape[-1])
    if t.dim() == 1:
        return 1, h, h
    if t.dim() == 2:
        return int(t.shape[0]), h, (t.stride(0) if t.shape[0] > 1 else h)
    if not t.is_contiguous():
        raise ValueError(f"{name} of more than two dimensions must be dense")
    return t.numel() // h, h, h


def mx_quantize(x, stream=None) -> MxTensor:
    """x [.., h] (float16 or bfloat16, h a multiple of 32) in MX."""
    torch = _torch()
    rows, h, ld = _as_rows(x, "x")
    if h % BLOCK != 0:
        raise ValueError(f"h = {h} must be a multiple of {BLOCK}")
    check_sizes("sgmv_mx_quantize", h)
    dt = dtype_code(x)
    handle = _stream_of(stream, x)
    lead = tuple(x.shape)[:-1]
    with _on(stream):
        codes = x.new_empty((*lead, h // 2), dtype=torch.uint8)
        scales = x.new_empty((*lead, h // BLOCK), dtype=torch.uint8)
    st = _lib.lib().sgmv_mx_quantize(handle, dt, codes.data_ptr(), scales.data_ptr(),
                                     x.data_ptr(), ld, rows, h)
    check(st, "sgmv_mx_quantize")
    return MxTensor(codes, scales)


def mx_dequantize(y, q: MxTensor, stream=None):
    """Write the values of ``q`` into y (float16 or bfloat16, the same shape), rounded once."""
    if tuple(y.shape) != tuple(q.shape):
        raise ValueError(f"y {tuple(y.shape)} does not match the values' {tuple(q.shape)}")
    rows, h, ld = _as_rows(y, "y")
    check_sizes("sgmv_mx_dequantize", h)
    dt = dtype_code(y)
    handle = _stream_of(stream, y, q.codes, q.scales)
    st = _lib.lib().sgmv_mx_dequantize(handle, dt, y.data_ptr(), ld,
                                       q.codes.data_ptr(), q.scales.data_ptr(), rows, h)
    check(st, "sgmv_mx_dequantize")
    return y


def mx_matmul(y, x, W: MxTensor, groups: Optional[RowGroups] = None, stream=None):
    """y[i] = x[i // share] @ W[g].T for the rows i of every group g, W [E, h_out, h_in] in MX
    (or [h_out, h_in] with ``groups=None``); rows of no group get zeros.  x is a tensor of
    y's dtype, or an MxTensor: then both sides of the product are in 4 bits."""
    n = y.shape[0]
    _check_rows(y, n, "y")
    E = 1 if groups is None else groups.n_groups
    shape = W.shape
    if len(shape) == 2:
        shape = (1, *shape)
    if len(shape) != 3 or shape[0] != E:
        raise ValueError(f"W must be [{E}, h_out, h_in]")
    _, h_out, h_in = shape
    xs = tuple(x.shape)
    if len(xs) != 2 or xs[1] != h_in or y.shape[1] != h_out:
        raise ValueError(f"x {xs} / y {tuple(y.shape)} do not match W's h_in = {h_in}, "
                         f"h_out = {h_out}")
    check_sizes("sgmv_mx_matmul", n, h_in, h_out)
    dt, share = dtype_code(y), _share(n, xs[0])
    if isinstance(x, MxTensor):
        starts, perm, E = _tables(groups, n, y)
        handle = _stream_of(stream, y, x.codes, x.scales, W.codes, W.scales)
        st = _lib.lib().sgmv_mx_matmul_quantized(
            handle, dt, y.data_ptr(), _ld(y), x.codes.data_ptr(), x.scales.data_ptr(), share,
            W.codes.data_ptr(), W.scales.data_ptr(), starts, perm, n, E, h_in, h_out)
        check(st, "sgmv_mx_matmul_quantized")
        return y
    _check_rows(x, xs[0], "x")
    if x.dtype != y.dtype:
        raise TypeError("x and y must share a dtype")
    starts, perm, E = _tables(groups, n, y)
    handle = _stream_of(stream, y, x, W.codes, W.scales)
    st = _lib.lib().sgmv_mx_matmul(
        handle, dt, y.data_ptr(), _ld(y), x.data_ptr(), _ld(x), share, W.codes.data_ptr(),
        W.scales.data_ptr(), starts, perm, n, E, h_in, h_out)
    check(st, "sgmv_mx_matmul")
    return y
