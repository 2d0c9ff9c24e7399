"""Plain fp64 definitions of routing to experts, of the weighted sum of a token's expert rows and of
their gradients, on numpy arrays.  Shares no code with the GPU path."""
from __future__ import annotations

import math

import numpy as np

INF = math.inf


def _exp(v: float) -> float:
    return math.exp(v) if v < 700 else INF


def scores_of(row, scores: str):
    """The score of every expert of one token, a list."""
    if scores == "sigmoid":
        return [math.nan if math.isnan(v) else 1.0 / (1.0 + _exp(-v)) if v > -700 else 0.0 for v in row]
    if any(math.isnan(v) or v == INF for v in row):
        return [math.nan] * len(row)
    top = max(row)
    if top == -INF:
        return [0.0] * len(row)
    e = [math.exp(v - top) for v in row]
    total = math.fsum(e)
    return [v / total for v in e]


def _rank(v: float):
    """Orders values, NaN above all."""
    return (1, 0.0) if math.isnan(v) else (0, v)


def _largest(values, count: int):
    """The places of the `count` largest, equal ones from the left; minus infinity is never taken."""
    at = [i for i, v in enumerate(values) if v != -INF]
    return sorted(at, key=lambda i: ((-_rank(values[i])[0], -_rank(values[i])[1]), i))[:count]


def choose(row, k, bias=None, scores="softmax", groups=1, keep=None, best=2):
    """The experts chosen for one token, at most k, in order."""
    row = [float(v) for v in row]
    keep = groups if keep is None else keep
    s = scores_of(row, scores)
    spoiled = scores == "softmax" and any(math.isnan(v) for v in s)
    if bias is None and (keep == groups or best == 1):
        c = [math.nan if spoiled else v for v in row]      # a score grows with its logit
    else:
        c = [v + (0.0 if bias is None else float(bias[i])) for i, v in enumerate(s)]
    c = [-INF if row[i] == -INF else v for i, v in enumerate(c)]
    if keep < groups:
        per = len(row) // groups
        total = []
        for g in range(groups):
            mine = c[g * per:(g + 1) * per]
            at = _largest(mine, best)
            total.append(math.fsum(mine[i] for i in at) if at and not any(math.isnan(mine[i]) for i in at)
                         else math.nan if at else -INF)
        stay = set(_largest(total, keep))
        c = [v if i // per in stay else -INF for i, v in enumerate(c)]
    return _largest(c, k)


def route(logits, k, bias=None, scores="softmax", groups=1, keep=None, best=2, normalize=True, scale=1.0):
    """(ids int32 [T, k], weights float64 [T, k])."""
    T = len(logits)
    ids, weights = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        row = [float(v) for v in logits[t]]
        at = choose(row, k, bias, scores, groups, keep, best)
        if at:
            ids[t, :len(at)] = at
            weights[t, :len(at)] = [scale * u for u in shares(row, at, scores, normalize)]
    return ids, weights


def shares(row, at, scores, normalize):
    """The scores of the experts `at`, over their sum with normalize (of scores too small for
    float64 as well, whose common factor is taken out first)."""
    s = scores_of(row, scores)
    if not normalize:
        return [s[i] for i in at]
    if any(math.isnan(s[i]) for i in at):
        return [math.nan] * len(at)
    top = max(row[i] for i in at)
    if scores == "softmax":
        e = [math.exp(row[i] - top) for i in at]
    else:
        low = min(top, 0.0)
        e = [1.0 / (1.0 + math.exp(-row[i])) if row[i] >= 0 else math.exp(row[i] - low) / (1.0 + math.exp(row[i]))
             for i in at]
    total = math.fsum(e)
    return [v / total for v in e]


def route_backward(logits, ids, dweights, scores="softmax", normalize=True, scale=1.0):
    """(dlogits float64 [T, E], magnitudes of the terms summed in them)."""
    T, E = np.shape(logits)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        row = [float(v) for v in logits[t]]
        places = [j for j, i in enumerate(ids[t]) if 0 <= i < E and row[i] != -INF]
        at = [int(ids[t][j]) for j in places]
        g = [scale * float(dweights[t][j]) for j in places]
        if not at:
            continue
        s = scores_of(row, scores)
        if scores == "softmax" and normalize:
            u = scores_of([row[i] for i in at], scores)        # of the chosen logits alone
        else:
            u = shares(row, at, scores, normalize)
        if scores == "softmax" and not normalize:
            inner = math.fsum(a * b for a, b in zip(g, u))
            size = math.fsum(abs(a * b) for a, b in zip(g, u))
            for i in range(E):
                if row[i] != -INF:
                    own = [g[m] for m in range(len(at)) if at[m] == i]
                    d[t, i] = s[i] * (math.fsum(own) - inner)
                    mag[t, i] = abs(s[i]) * (math.fsum(abs(v) for v in own) + size)
            continue
        inner = math.fsum(a * b for a, b in zip(g, u)) if normalize else 0.0
        size = math.fsum(abs(a * b) for a, b in zip(g, u)) if normalize else 0.0
        for m, i in enumerate(at):
            rest = 1.0 if scores == "softmax" else 1.0 / (1.0 + _exp(row[i]))
            d[t, i] += u[m] * rest * (g[m] - inner)
            mag[t, i] += abs(u[m]) * rest * (abs(g[m]) + size)
    return d, mag


def combine(y, weights, k):
    """(out [T, h], magnitudes): out[t] = sum over j of weights[t, j] y[t * k + j]."""
    p = y.reshape(-1, k, y.shape[1]) * (1.0 if weights is None else weights[:, :, None])
    return p.sum(1), np.abs(p).sum(1)


def combine_backward(dout, y, weights, k):
    """(dy [T * k, h], dweights [T, k] or None, magnitudes of dweights)."""
    T, h = dout.shape
    if weights is None:
        return np.repeat(dout, k, 0), None, None
    dy = (weights[:, :, None] * dout[:, None, :]).reshape(T * k, h)
    p = y.reshape(T, k, h) * dout[:, None, :]
    return dy, p.sum(2), np.abs(p).sum(2)
