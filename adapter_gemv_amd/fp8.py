"""8-bit floating point with a scale for each block of 128 on torch tensors: quantisation, products
with both sides in it, and the gradient of their rows.  Argument checks and marshalling only
(``sgmv_block_*`` in include/sgmv.h, which defines the format)::

    Wq = fp8_quantize_weight(W)             # W [.., h_out, h_in]; or Fp8Weight(codes, scales)
    fp8_matmul(y, x, Wq, groups)            # y[i] = x8[i // share] @ Wq[g].T, x taken to 8 bits
    fp8_matmul_dx(dx, dy, Wq, groups)       # dx[i] = dy8[i] @ Wq[g]
    fp8_dequantize(W, Wq)                   # the values back, in W's type

The gradient of the weights is ``group_matmul_dw``, of the 16-bit rows.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

from . import _lib
from ._lib import check, check_sizes
from .grouped import RowGroups, _empty, _matrix, _share, _stream_of, _tables
from .mx import _as_rows
from .sgmv import _torch, dtype_code

BLOCK = 128


def _blocks(h: int) -> int:
    return (h + BLOCK - 1) // BLOCK


def _made(kind, codes, scales):
    """A value of parts that need no check."""
    q = object.__new__(kind)
    q.codes, q.scales = codes, scales
    return q


def _check_parts(codes, scales, shape):
    torch = _torch()
    if codes.dtype is not torch.float8_e4m3fn or scales.dtype is not torch.float32:
        raise TypeError("codes must be float8_e4m3fn and scales float32")
    if scales.shape != shape:
        raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} do not match: "
                         f"scales must be {shape}")
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("codes and scales must be dense")


@dataclasses.dataclass
class Fp8Rows:
    """``codes`` float8_e4m3fn [.., h] and ``scales`` float32 [.., ceil(h / 128)], both dense."""
    codes: object
    scales: object

    def __post_init__(self):
        c = self.codes
        if c.dim() < 1:
            raise ValueError("codes must be [.., h]")
        s = c.shape
        _check_parts(c, self.scales, (*s[:-1], _blocks(s[-1])))

    @property
    def shape(self):
        """The shape of the values."""
        return tuple(self.codes.shape)


@dataclasses.dataclass
class Fp8Weight:
    """``codes`` float8_e4m3fn [E, h_out, h_in] and ``scales`` float32 [E, ceil(h_out / 128),
    ceil(h_in / 128)] (or both without E), dense."""
    codes: object
    scales: object

    def __post_init__(self):
        c = self.codes
        if c.dim() not in (2, 3):
            raise ValueError("codes must be [E, h_out, h_in] or [h_out, h_in]")
        s = c.shape
        _check_parts(c, self.scales, (*s[:-2], _blocks(s[-2]), _blocks(s[-1])))

    @property
    def shape(self):
        """The shape of the values."""
        return tuple(self.codes.shape)


def _weight_groups(W, name: str):
    """(E, h_out, h_in, elements between groups) of a 16-bit weight."""
    if W.dim() not in (2, 3):
        raise ValueError(f"{name} must be [E, h_out, h_in] or [h_out, h_in]")
    E = int(W.shape[0]) if W.dim() == 3 else 1
    h_out, h_in = int(W.shape[-2]), int(W.shape[-1])
    if W.numel() and ((W.stride(-1) != 1 and h_in > 1) or (W.stride(-2) != h_in and h_out > 1)):
        raise ValueError(f"{name} must hold dense row-major groups")
    return E, h_out, h_in, (W.stride(0) if E > 1 else h_out * h_in)


def fp8_quantize(x, stream=None) -> Fp8Rows:
    """x [.., h] (float16 or bfloat16, h a multiple of 16) in 8 bits, one scale for 128 elements."""
    torch = _torch()
    rows, h, ld = _as_rows(x, "x")
    check_sizes("sgmv_block_quantize", h)
    dt = dtype_code(x)
    handle = _stream_of(stream, x)
    codes = _empty(x, x.shape, torch.float8_e4m3fn, stream)
    scales = _empty(x, (*x.shape[:-1], _blocks(h)), torch.float32, stream)
    st = _lib.lib().sgmv_block_quantize(handle, dt, codes.data_ptr(), scales.data_ptr(), x.data_ptr(), ld, rows, h)
    check(st, "sgmv_block_quantize")
    return _made(Fp8Rows, codes, scales)


def fp8_quantize_weight(W, stream=None) -> Fp8Weight:
    """W [E, h_out, h_in] or [h_out, h_in] (float16 or bfloat16, h_in a multiple of 16, h_out of 8) in
    8 bits, one scale for 128 x 128 elements."""
    torch = _torch()
    E, h_out, h_in, stride = _weight_groups(W, "W")
    check_sizes("sgmv_block_quantize_weight", E, h_out, h_in)
    dt = dtype_code(W)
    handle = _stream_of(stream, W)
    codes = _empty(W, W.shape, torch.float8_e4m3fn, stream)
    scales = _empty(W, (*W.shape[:-2], _blocks(h_out), _blocks(h_in)), torch.float32, stream)
    st = _lib.lib().sgmv_block_quantize_weight(handle, dt, codes.data_ptr(), scales.data_ptr(), W.data_ptr(), stride,
                                             E, h_in, h_out)
    check(st, "sgmv_block_quantize_weight")
    return _made(Fp8Weight, codes, scales)


def fp8_dequantize(y, q, stream=None):
    """Write the values of ``q`` (Fp8Rows or Fp8Weight) into y (float16 or bfloat16, the same
    shape), rounded once."""
    if tuple(y.shape) != q.shape:
        raise ValueError(f"y {tuple(y.shape)} does not match the values' {q.shape}")
    dt = dtype_code(y)
    if isinstance(q, Fp8Weight):
        E, h_out, h_in, stride = _weight_groups(y, "y")
        check_sizes("sgmv_block_dequantize_weight", E, h_out, h_in)
        handle = _stream_of(stream, y, q.codes, q.scales)
        st = _lib.lib().sgmv_block_dequantize_weight(handle, dt, y.data_ptr(), stride, q.codes.data_ptr(),
                                                   q.scales.data_ptr(), E, h_in, h_out)
        check(st, "sgmv_block_dequantize_weight")
        return y
    rows, h, ld = _as_rows(y, "y")
    check_sizes("sgmv_block_dequantize", h)
    handle = _stream_of(stream, y, q.codes, q.scales)
    st = _lib.lib().sgmv_block_dequantize(handle, dt, y.data_ptr(), ld, q.codes.data_ptr(), q.scales.data_ptr(),
                                        rows, h)
    check(st, "sgmv_block_dequantize")
    return y


def _product(out, rows, W: Fp8Weight, groups: Optional[RowGroups], stream, dx: bool):
    where = "sgmv_block_matmul_dx" if dx else "sgmv_block_matmul"
    n, out_cols, ld_out = _matrix(out, "dx" if dx else "y")
    E = 1 if groups is None else groups.n_groups
    codes, scales = W.codes, W.scales
    shape = codes.shape
    h_out, h_in = shape[-2:]
    if (shape[0] if len(shape) == 3 else 1) != E:
        raise ValueError(f"W must be [{E}, h_out, h_in]")
    depth, cols = (h_out, h_in) if dx else (h_in, h_out)
    eight = isinstance(rows, Fp8Rows)
    if eight:
        rs = rows.codes.shape
        if len(rs) != 2:
            raise ValueError("rows in 8 bits must be [n, h]")
    else:
        *rs, ld = _matrix(rows, "dy" if dx else "x")
    if rs[1] != depth or out_cols != cols:
        raise ValueError(f"rows {tuple(rs)} and output {tuple(out.shape)} do not match W's h_in = {h_in}, "
                         f"h_out = {h_out}")
    if dx and rs[0] != n:
        raise ValueError(f"dy has {rs[0]} rows, dx {n}")
    check_sizes(where, n, h_in, h_out)
    dt, share = dtype_code(out), _share(n, rs[0])
    starts, perm, E = _tables(groups, n, out)
    lib = _lib.lib()
    tail = (codes.data_ptr(), scales.data_ptr(), starts, perm, n, E, h_in, h_out)
    if eight:
        handle = _stream_of(stream, out, rows.codes, rows.scales, codes, scales)
        head = (handle, dt, out.data_ptr(), ld_out, rows.codes.data_ptr(), rows.scales.data_ptr())
        st = (lib.sgmv_block_matmul_dx_quantized(*head, *tail) if dx else
              lib.sgmv_block_matmul_quantized(*head, share, *tail))
        check(st, where + "_quantized")
        return out
    if rows.dtype is not out.dtype:
        raise TypeError("the rows and the output must share a dtype")
    handle = _stream_of(stream, out, rows, codes, scales)
    room = (lib.sgmv_block_dx_workspace_bytes(n, h_out) if dx else
            lib.sgmv_block_workspace_bytes(n, share, E, starts is not None, h_in, h_out))
    at = None
    if room:
        space = _empty(out, (room,), _torch().uint8, stream)
        at = space.data_ptr()
    head = (handle, dt, out.data_ptr(), ld_out, rows.data_ptr(), ld)
    st = (lib.sgmv_block_matmul_dx(*head, *tail, at, room) if dx else
          lib.sgmv_block_matmul(*head, share, *tail, at, room))
    check(st, where)
    return out


def fp8_matmul(y, x, W: Fp8Weight, groups: Optional[RowGroups] = None, stream=None):
    """y[i] = x[i // share] @ W[g].T for the rows i of every group g (``groups=None``: one W); rows of
    no group get zeros.  x is a tensor of y's dtype, taken to 8 bits within the call, or an Fp8Rows."""
    return _product(y, x, W, groups, stream, False)


def fp8_matmul_dx(dx, dy, W: Fp8Weight, groups: Optional[RowGroups] = None, stream=None):
    """dx[i] = dy[i] @ W[g] for the rows i of every group g; rows of no group get zeros.  dy is a
    tensor of dx's dtype, taken to 8 bits along h_out within the call, or an Fp8Rows.  Where rows
    share an x, its gradient is the sum of theirs (``combine_rows``)."""
    return _product(dx, dy, W, groups, stream, True)
