"""Routing to experts, and the weighted sum of each token's expert rows, with their gradients, on
torch tensors.

Argument checks and marshalling only (``sgmv_route*`` and ``sgmv_combine_rows*`` in
include/sgmv.h).  Around the products grouped by expert, forwards and back::

    routes = route(logits, k)                            # logits [T, E]
    groups = group_rows(routes.ids.view(-1), E)
    group_matmul(y, x, W, groups)                        # y [T * k, h]
    combine_rows(out, y, routes.weights)                 # out[t] = sum_j weights[t, j] y[t * k + j]

    combine_rows_backward(dy, dweights, dout, y, routes.weights)
    group_matmul_dx(dxs, dy, W, groups)
    combine_rows(dx, dxs)                                # a row's k gradients summed
    route_backward(dlogits, dweights, logits, routes)
"""
from __future__ import annotations

import dataclasses
from typing import Optional

from . import _lib
from ._lib import check, check_sizes
from .grouped import _empty, _matrix, _stream_of
from .sgmv import _torch, dtype_code

SCORES = {"softmax": _lib.SOFTMAX, "sigmoid": _lib.SIGMOID}


@dataclasses.dataclass
class Routes:
    """The experts of each token, ``ids`` int32 [T, k] (-1: none), their ``weights`` float32
    [T, k], and how these were made of the scores."""
    ids: object
    weights: object
    scores: str = "softmax"
    normalize: bool = True
    scale: float = 1.0


def _logits(t, name: str):
    """(T, E, elements between rows, dtype) of logits."""
    shape = t.shape
    if len(shape) != 2 or shape[1] == 0:
        raise ValueError(f"{name} must be [T, E]")
    dt = _lib.F32 if t.dtype is _torch().float32 else dtype_code(t)
    T, E = shape
    row, column = t.stride()
    if column != 1 and E > 1:
        raise ValueError(f"{name} must have unit column stride")
    return T, E, row if T > 1 else E, dt


def _scores_code(scores: str) -> int:
    if scores not in SCORES:
        raise ValueError(f"scores must be one of {', '.join(SCORES)}")
    return SCORES[scores]


def _dense(t, dtype, shape, name: str):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a dense {str(dtype).split('.')[-1]} tensor {list(shape)}")


def route(logits, k: int, *, bias=None, scores: str = "softmax", expert_groups: int = 1,
          keep_groups: Optional[int] = None, group_best: int = 2, normalize: bool = True,
          scale: float = 1.0, stream=None) -> Routes:
    """The k experts of each token by its logits [T, E] (float32, float16 or bfloat16).

    ``scores`` of the logits, plus ``bias`` (float32 [E], for the choice alone), choose: of the
    ``expert_groups`` equal runs of experts the ``keep_groups`` (all) whose ``group_best`` (1 or 2)
    best experts sum up highest, and of their experts the k best.  The weights are ``scale`` times
    the scores, divided by the sum of the chosen ones with ``normalize``.  A token whose logits are all
    minus infinity gets ids -1 and weights 0."""
    torch = _torch()
    (T, E, ld, dt), code = _logits(logits, "logits"), _scores_code(scores)
    keep = expert_groups if keep_groups is None else keep_groups
    check_sizes("sgmv_route", T, E, k, expert_groups, keep, group_best)
    if k < 1 or k > E:
        check(_lib.ERR_SHAPE, "sgmv_route")
    if bias is not None:
        _dense(bias, torch.float32, (E,), "bias")
        handle = _stream_of(stream, logits, bias)
    else:
        handle = _stream_of(stream, logits)
    ids = _empty(logits, (T, k), torch.int32, stream)
    weights = _empty(logits, (T, k), torch.float32, stream)
    st = _lib.lib().sgmv_route(handle, dt, ids.data_ptr(), weights.data_ptr(), logits.data_ptr(),
                               ld, None if bias is None else bias.data_ptr(), T, E, k,
                               expert_groups, keep, group_best, code, bool(normalize), scale)
    check(st, "sgmv_route")
    return Routes(ids, weights, scores, bool(normalize), float(scale))


def route_backward(dlogits, dweights, logits, routes: Routes, stream=None):
    """Write the gradient of the logits into ``dlogits`` (their shape and type) from that of the
    weights (float32 [T, k]); the choice of experts is held fixed."""
    torch = _torch()
    (T, E, ld, dt), code = _logits(logits, "logits"), _scores_code(routes.scores)
    dT, dE, ld_d, ddt = _logits(dlogits, "dlogits")
    if ddt != dt:
        raise TypeError("logits and dlogits must share a dtype")
    if dT != T or dE != E:
        raise ValueError(f"dlogits {tuple(dlogits.shape)} does not match logits [{T}, {E}]")
    ids = routes.ids
    if ids.dim() != 2:
        raise ValueError(f"routes.ids must be [{T}, k]")
    k = int(ids.shape[1])
    _dense(ids, torch.int32, (T, k), "routes.ids")
    _dense(dweights, torch.float32, (T, k), "dweights")
    check_sizes("sgmv_route_backward", T, E)
    handle = _stream_of(stream, dlogits, dweights, logits, ids)
    st = _lib.lib().sgmv_route_backward(handle, dt, dlogits.data_ptr(), ld_d, dweights.data_ptr(),
                                        logits.data_ptr(), ld, ids.data_ptr(), T, E, k, code,
                                        bool(routes.normalize), routes.scale)
    check(st, "sgmv_route_backward")
    return dlogits


def _tokens(out, y, weights, what: str):
    """(T, k, h, dtype, strides of out and y) of a call whose rows are y [T * k, h] and whose tokens are
    out [T, h]."""
    T, h, ld_out = _matrix(out, what)
    n, width, ld_y = _matrix(y, "the experts' rows")
    if width != h:
        raise ValueError(f"{what} [., {h}] and the experts' rows [., {width}] do not match")
    if out.dtype is not y.dtype:
        raise TypeError("all rows must share a dtype")
    k = n // T if T else 1
    if weights is not None:
        if not T and weights.dim() == 2:
            k = weights.shape[1]
        _dense(weights, _torch().float32, (T, k), "weights")
    if n != T * k or k < 1:
        raise ValueError(f"{n} rows are not the experts' of {T} tokens")
    check_sizes("sgmv_combine_rows", n, k, h)
    return T, k, h, dtype_code(y), ld_out, ld_y


def combine_rows(out, y, weights=None, add: bool = False, stream=None):
    """out[t] = sum over j of weights[t, j] * y[t * k + j] (plus what out holds, with ``add``);
    without weights their plain sum.  out [T, h], y [T * k, h], weights float32 [T, k]."""
    T, k, h, dt, ld_out, ld_y = _tokens(out, y, weights, "out")
    if weights is None:
        handle, at = _stream_of(stream, out, y), None
    else:
        handle, at = _stream_of(stream, out, y, weights), weights.data_ptr()
    st = _lib.lib().sgmv_combine_rows(handle, dt, out.data_ptr(), ld_out, y.data_ptr(), ld_y, at, T, k, h, bool(add))
    check(st, "sgmv_combine_rows")
    return out


def combine_rows_backward(dy, dweights, dout, y=None, weights=None, stream=None):
    """dy[t * k + j] = weights[t, j] * dout[t] and dweights[t, j] = dout[t] . y[t * k + j]; without
    weights (then dweights and y are None) dout's rows alone, k times each."""
    T, k, h, dt, ld_dout, ld_dy = _tokens(dout, dy, weights, "dout")
    if weights is None:
        if dweights is not None:
            raise ValueError("dweights without weights")
        handle = _stream_of(stream, dy, dout)
        st = _lib.lib().sgmv_combine_rows_backward(handle, dt, dy.data_ptr(), ld_dy, None, dout.data_ptr(), ld_dout,
                                                   None, 0, None, T, k, h)
    else:
        _dense(dweights, _torch().float32, (T, k), "dweights")
        n, width, ld_y = _matrix(y, "y")
        if n != T * k or width != h:
            raise ValueError(f"y [{n}, {width}] does not match dy [{T * k}, {h}]")
        if y.dtype is not dy.dtype:
            raise TypeError("all rows must share a dtype")
        handle = _stream_of(stream, dy, dweights, dout, y, weights)
        st = _lib.lib().sgmv_combine_rows_backward(handle, dt, dy.data_ptr(), ld_dy, dweights.data_ptr(),
                                                   dout.data_ptr(), ld_dout, y.data_ptr(), ld_y, weights.data_ptr(),
                                                   T, k, h)
    check(st, "sgmv_combine_rows_backward")
    return dy, dweights
