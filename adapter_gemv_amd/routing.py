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
from .grouped import _empty, _ld, _stream_of
from .sgmv import _check_rows, _torch, dtype_code

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


def _logits_code(t, name: str) -> int:
    if t.dim() != 2 or not t.is_contiguous() and t.stride(1) != 1 and t.shape[1] > 1 or t.shape[1] == 0:
        raise ValueError(f"{name} must be [T, E] with unit column stride")
    return _lib.F32 if t.dtype is _torch().float32 else dtype_code(t)


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
    dt, code = _logits_code(logits, "logits"), _scores_code(scores)
    T, E = logits.shape
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
                               _ld(logits), None if bias is None else bias.data_ptr(), T, E, k,
                               expert_groups, keep, group_best, code, bool(normalize), scale)
    check(st, "sgmv_route")
    return Routes(ids, weights, scores, bool(normalize), float(scale))


def route_backward(dlogits, dweights, logits, routes: Routes, stream=None):
    """Write the gradient of the logits into ``dlogits`` (their shape and type) from that of the
    weights (float32 [T, k]); the choice of experts is held fixed."""
    torch = _torch()
    dt, code = _logits_code(logits, "logits"), _scores_code(routes.scores)
    if _logits_code(dlogits, "dlogits") != dt:
        raise TypeError("logits and dlogits must share a dtype")
    T, E = logits.shape
    if tuple(dlogits.shape) != (T, E):
        raise ValueError(f"dlogits {tuple(dlogits.shape)} does not match logits [{T}, {E}]")
    ids = routes.ids
    if ids.dim() != 2:
        raise ValueError(f"routes.ids must be [{T}, k]")
    k = int(ids.shape[1])
    _dense(ids, torch.int32, (T, k), "routes.ids")
    _dense(dweights, torch.float32, (T, k), "dweights")
    check_sizes("sgmv_route_backward", T, E)
    handle = _stream_of(stream, dlogits, dweights, logits, ids)
    st = _lib.lib().sgmv_route_backward(handle, dt, dlogits.data_ptr(), _ld(dlogits), dweights.data_ptr(),
                                        logits.data_ptr(), _ld(logits), ids.data_ptr(), T, E, k, code,
                                        bool(routes.normalize), routes.scale)
    check(st, "sgmv_route_backward")
    return dlogits


def _tokens(out, y, weights, what: str):
    """(T, k, h, dtype) of a call whose rows are y [T * k, h] and whose tokens are out [T, h]."""
    if out.dim() != 2 or y.dim() != 2:
        raise ValueError(f"{what} and the experts' rows must be matrices")
    (T, h), (n, width) = out.shape, y.shape
    _check_rows(out, T, what)
    _check_rows(y, n, "the experts' rows")
    if width != h:
        raise ValueError(f"{what} [., {h}] and the experts' rows [., {width}] do not match")
    if out.dtype is not y.dtype:
        raise TypeError("all rows must share a dtype")
    k = n // T if T else 1
    if weights is not None:
        if weights.dim() != 2:
            raise ValueError(f"weights must be [{T}, k]")
        if not T:
            k = weights.shape[1]
        _dense(weights, _torch().float32, (T, k), "weights")
    if n != T * k or k < 1:
        raise ValueError(f"{n} rows are not the experts' of {T} tokens")
    check_sizes("sgmv_combine_rows", n, k, h)
    return T, k, h, dtype_code(y)


def combine_rows(out, y, weights=None, add: bool = False, stream=None):
    """out[t] = sum over j of weights[t, j] * y[t * k + j] (plus what out holds, with ``add``);
    without weights their plain sum.  out [T, h], y [T * k, h], weights float32 [T, k]."""
    T, k, h, dt = _tokens(out, y, weights, "out")
    handle = _stream_of(stream, out, y) if weights is None else _stream_of(stream, out, y, weights)
    st = _lib.lib().sgmv_combine_rows(handle, dt, out.data_ptr(), _ld(out), y.data_ptr(), _ld(y),
                                      None if weights is None else weights.data_ptr(), T, k, h, bool(add))
    check(st, "sgmv_combine_rows")
    return out


def combine_rows_backward(dy, dweights, dout, y=None, weights=None, stream=None):
    """dy[t * k + j] = weights[t, j] * dout[t] and dweights[t, j] = dout[t] . y[t * k + j]; without
    weights (then dweights and y are None) dout's rows alone, k times each."""
    T, k, h, dt = _tokens(dout, dy, weights, "dout")
    if weights is None:
        if dweights is not None:
            raise ValueError("dweights without weights")
        handle = _stream_of(stream, dy, dout)
        st = _lib.lib().sgmv_combine_rows_backward(handle, dt, dy.data_ptr(), _ld(dy), None, dout.data_ptr(),
                                                   _ld(dout), None, 0, None, T, k, h)
    else:
        _dense(dweights, _torch().float32, (T, k), "dweights")
        _check_rows(y, T * k, "y")
        if y.shape[1] != h:
            raise ValueError(f"y [., {y.shape[1]}] does not match dout [., {h}]")
        if y.dtype != dy.dtype:
            raise TypeError("all rows must share a dtype")
        handle = _stream_of(stream, dy, dweights, dout, y, weights)
        st = _lib.lib().sgmv_combine_rows_backward(handle, dt, dy.data_ptr(), _ld(dy), dweights.data_ptr(),
                                                   dout.data_ptr(), _ld(dout), y.data_ptr(), _ld(y),
                                                   weights.data_ptr(), T, k, h)
    check(st, "sgmv_combine_rows_backward")
    return dy, dweights
