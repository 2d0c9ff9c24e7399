"""Routing to experts, combining their rows, and 8-bit products with a scale for each block of 128:
cases, plain forms and 64-bit values.

A case names one pass through one operator:

* ``route``          logits to the ids and weights of each token's experts: softmax or sigmoid scores,
                     a bias for the choice alone, expert groups of which the best stay, the k best
                     experts of these (ties: the lowest), weights renormalised or not;
* ``route_train``    the same, and the gradient of the logits from that of the weights;
* ``combine``        the rows of each token's experts summed with its weights;
* ``combine_train``  the same, and the gradients of the rows and of the weights;
* ``quantize``       a 16-bit weight to 8-bit floating point (four exponent and three mantissa bits,
                     one power of two for each 128 x 128) and back;
* ``fp8``            16-bit rows, taken to 8 bits within the call (one power of two for each 128
                     elements of a row), times weights held in 8 bits, dense or by expert;
* ``fp8_train``      a weight taken to 8 bits, that product, and the gradient of its rows.

A token whose logits are all minus infinity is padding: it gets no expert (id -1, weight 0).  Rows with
a negative id belong to no expert: their output rows are zero.
"""
import math
import random

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BLOCK = 128
MOST = 448.0  # the largest 8-bit value


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def _route(op, dtype, tokens, experts, k, scores="softmax", bias=False, groups=1, keep=1, best=1,
           normalize=True, scale=1.0, padded=0.0):
    return {"op": op, "dtype": dtype, "tokens": tokens, "experts": experts, "k": k, "scores": scores,
            "bias": bias, "groups": groups, "keep": keep, "best": best, "normalize": normalize,
            "scale": scale, "padded": padded}


def _combine(op, dtype, tokens, k, h):
    return {"op": op, "dtype": dtype, "tokens": tokens, "k": k, "h": h}


def _product(op, dtype, tokens, top_k, experts, h_in, h_out, skew=0.0, away=0.0):
    return {"op": op, "dtype": dtype, "tokens": tokens, "top_k": top_k, "experts": experts,
            "h_in": h_in, "h_out": h_out, "skew": skew, "away": away}


def listed():
    cases = {
        # one generated token over a small expert layer: latency
        "route_one_token": _route("route", "bf16", 1, 64, 2),
        # prompts over many experts in groups, a balancing bias, a few padded tokens
        "route_prompts": _route("route", "f32", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5, 0.02),
        # a small training step of few experts, weights as softmax left them, odd sizes
        "route_train_small": _route("route_train", "f16", 777, 60, 4, normalize=False),
        # a training step of full length
        "route_train": _route("route_train", "f32", 16384, 128, 8, "sigmoid", True),
        # a decode batch's expert rows
        "combine_decode": _combine("combine", "f16", 32, 2, 4096),
        # a training step's expert rows, odd length
        "combine_train": _combine("combine_train", "bf16", 8191, 4, 5120),
        # the feed-forward weights of some experts, once when they are loaded
        "quantize_weight": _product("quantize", "bf16", 0, 0, 4, 8192, 14336),
        # one generated token through a dense projection
        "fp8_one_token": _product("fp8", "bf16", 1, 1, 1, 4096, 4096),
        # a decode batch over many narrow experts
        "fp8_experts_decode": _product("fp8", "f16", 32, 2, 64, 4096, 1024, 0.3),
        # a prompt of odd length through wide experts, some popular
        "fp8_experts_prompt": _product("fp8", "bf16", 1531, 2, 8, 5120, 13824, 0.6),
        # a small training step: ragged, blocks that end early, a tenth of the rows held elsewhere
        "fp8_train_small": _product("fp8_train", "f16", 777, 2, 4, 1040, 528, 0.6, 0.1),
        # a training step of full width
        "fp8_train": _product("fp8_train", "bf16", 8192, 2, 16, 4096, 4096, 0.3),
    }
    return [{"name": name, **case} for name, case in cases.items()]


def _log(rng, lo, hi, unit=1):
    return max(unit, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit)) * unit)


def draw(rng):
    top = [work(c) for c in listed()]
    most = {key: max(w[key] for w in top) for key in ("bytes", "flops")}
    while True:
        op = rng.choice(["route", "route", "route_train", "route_train", "combine", "combine_train",
                         "quantize", "fp8", "fp8", "fp8_train", "fp8_train"])
        dtype = rng.choice(["bf16", "f16", "f32"] if op.startswith("route") else ["bf16", "f16"])
        if op.startswith("route"):
            groups = rng.choice([1, 1, 2, 4, 8])
            each = _log(rng, 4 if groups == 1 else 2, 512 // groups)
            keep = rng.randint(1, groups)
            scores = rng.choice(["softmax", "sigmoid"])
            c = _route(op, dtype, _log(rng, 1, 20000), groups * each, rng.randint(1, min(12, keep * each)),
                       scores, rng.random() < 0.5, groups, keep, rng.choice([1, 2]), rng.random() < 0.6,
                       rng.choice([1.0, 2.5]), rng.choice([0.0, 0.05]))
        elif op.startswith("combine"):
            c = _combine(op, dtype, _log(rng, 1, 16000), rng.randint(1, 8), _log(rng, 256, 8192, 8))
        elif op == "quantize":
            c = _product(op, dtype, 0, 0, rng.randint(1, 8), _log(rng, 256, 14336, 16), _log(rng, 256, 14336, 16))
        else:
            experts = 1 if rng.random() < 0.3 else _log(rng, 2, 96)
            c = _product(op, dtype, _log(rng, 64 if op == "fp8_train" else 1, 12000),
                         rng.randint(1, min(6, experts)), experts, _log(rng, 256, 14336, 16),
                         _log(rng, 256, 14336, 16), rng.choice([0.0, 0.3, 0.6, 1.0]),
                         rng.choice([0.0, 0.0, 0.25]) if experts > 1 else 0.0)
            if experts * c["h_in"] * c["h_out"] > 6e8:
                continue
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _popularity(case):
    p = [(e + 1.0) ** -case["skew"] for e in range(case["experts"])]
    return [v / sum(p) for v in p]


def work(case):
    op = case["op"]
    if op.startswith("route"):
        rows, one = case["tokens"] * case["experts"], 4 if case["dtype"] == "f32" else 2
        chosen = case["tokens"] * case["k"]
        # logits in, ids and weights out; training: the weights' gradient in, the logits' out
        if op == "route":
            return {"bytes": one * rows + 8 * chosen, "flops": 4 * rows}
        return {"bytes": 2 * one * rows + 12 * chosen, "flops": 8 * rows}
    if op.startswith("combine"):
        n, y = case["tokens"], case["tokens"] * case["k"] * case["h"]
        if op == "combine":
            return {"bytes": 2 * y + 2 * n * case["h"] + 4 * n * case["k"], "flops": 2 * y}
        # rows, out's gradient and weights in; out and both gradients out
        return {"bytes": 4 * y + 4 * n * case["h"] + 8 * n * case["k"], "flops": 5 * y}
    weight = case["h_in"] * case["h_out"]
    if op == "quantize":
        return {"bytes": 4 * case["experts"] * weight, "flops": 2 * case["experts"] * weight}
    n = case["tokens"] * case["top_k"]
    here = n * (1.0 - case["away"])
    x, y = 2 * case["tokens"] * case["h_in"], 2 * n * case["h_out"]
    flops = 2.0 * here * weight
    if op == "fp8":
        met = sum(1.0 - (1.0 - p) ** here for p in _popularity(case))
        return {"bytes": x + y + met * weight, "flops": flops}
    # x, y's gradient and the 16-bit weight in; y and a gradient for each row out
    return {"bytes": x + 2 * y + 2 * n * case["h_in"] + 2 * case["experts"] * weight, "flops": 2 * flops}


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _ids(case, gen):
    """int32 [tokens * top_k]: every token's experts, all different, the popular ones more often."""
    p = torch.tensor(_popularity(case), dtype=torch.float32, device="cuda")
    noise = torch.rand(case["tokens"], case["experts"], generator=gen, device="cuda")
    score = torch.log(p) - torch.log(-torch.log(noise.clamp(1e-9, 1 - 1e-7)))
    ids = torch.topk(score, case["top_k"], dim=1).indices.to(torch.int32).reshape(-1)
    if case["away"]:
        gone = torch.rand(ids.shape, generator=gen, device="cuda") < case["away"]
        ids = torch.where(gone, torch.full_like(ids, -1), ids)
    return ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * std

    if op.startswith("route"):
        # a trained layer's logits: experts of different popularity, tokens that care more or less
        T, E = case["tokens"], case["experts"]
        logits = normal(T, E, std=1.5) * torch.exp(normal(T, 1, std=0.3)) + normal(E, std=0.5)
        if case["padded"]:
            logits[torch.rand(T, generator=gen, device="cuda") < case["padded"]] = -math.inf
        s = {"case": case, "logits": logits.to(t), "bias": normal(E, std=0.1) if case["bias"] else None}
        if op == "route_train":
            s["dweights"] = normal(T, case["k"])
        return s
    if op.startswith("combine"):
        T, k, h = case["tokens"], case["k"], case["h"]
        s = {"case": case, "y": normal(T * k, h).to(t), "weights": torch.softmax(normal(T, k), 1)}
        if op == "combine_train":
            s["dout"] = normal(T, h).to(t)
        return s
    E, K, N = case["experts"], case["h_in"], case["h_out"]
    if op == "quantize":
        # rows and columns of different size
        W = normal(E, N, K, std=K ** -0.5)
        W *= torch.exp(normal(E, N, 1, std=0.5))
        W[:, :, torch.randperm(K, generator=gen, device="cuda")[: K // 128 + 1]] *= 8.0
        return {"case": case, "W": W.to(t)}
    x = normal(case["tokens"], K) * torch.exp(normal(case["tokens"], 1, std=0.5))
    s = {"case": case, "x": x.to(t), "ids": _ids(case, gen) if E > 1 else None}
    W = normal(E, N, K, std=K ** -0.5)
    if op == "fp8":
        # a checkpoint's weights: scales of any value, each block's largest element at the top
        s["codes"], s["scales"] = _checkpoint(W)
        return s
    s["W"] = W.to(t)
    s["dy"] = normal(case["tokens"] * case["top_k"], N, std=N ** -0.5).to(t)
    return s


def _padded(v, *dims):
    """v with zeros up to whole blocks in these dimensions (the last ones)."""
    pad = []
    for d in reversed(dims):
        pad += [0, -v.shape[d] % BLOCK]
    return torch.nn.functional.pad(v, pad) if any(pad) else v


def _checkpoint(W):
    E, N, K = W.shape
    v = _padded(W, -2, -1).unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK))
    scales = v.abs().amax((2, 4)) / MOST
    v = v / scales[:, :, None, :, None]
    codes = v.clamp_(-MOST, MOST).flatten(3, 4).flatten(1, 2)[:, :N, :K].contiguous().to(torch.float8_e4m3fn)
    return codes, scales


# --------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------
def _scores(logits, scores):
    """Scores in 64 bits: values next to each other decide which experts are chosen."""
    v = logits.double()
    if scores == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-v))
    e = torch.exp(v - v.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    c = s["case"]
    logits, E, k, G = s["logits"], c["experts"], c["k"], c["groups"]
    score = _scores(logits, c["scores"])
    out = logits == -math.inf
    choice = score if s["bias"] is None else score + s["bias"].double()
    choice = torch.where(out, torch.full_like(choice, -math.inf), choice)
    if c["keep"] < G:
        best = torch.sort(choice.unflatten(1, (G, E // G)), dim=2, descending=True).values[:, :, : c["best"]]
        some = best[:, :, :1] > -math.inf
        group = torch.where(best > -math.inf, best, torch.zeros_like(best)).sum(2)
        group = torch.where(some[:, :, 0], group, torch.full_like(group, -math.inf))
        kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        keep = torch.zeros_like(group, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep.repeat_interleave(E // G, 1), choice, torch.full_like(choice, -math.inf))
    value, ids = torch.sort(choice, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    none = value == -math.inf
    picked = torch.where(none, torch.zeros_like(value), torch.gather(score, 1, ids))
    total = picked.sum(1, keepdim=True) if c["normalize"] else 1.0
    weights = torch.where(none, torch.zeros_like(picked), picked / total * c["scale"])
    result = {"ids": torch.where(none, torch.full_like(ids, -1), ids).to(torch.int32), "weights": weights.float()}
    if c["op"] == "route":
        return result
    g = torch.where(none, torch.zeros_like(picked), s["dweights"].double() * c["scale"])
    u = torch.where(none, torch.zeros_like(picked), picked / total)
    dl = torch.zeros_like(score)
    if c["normalize"]:
        d = u * (g - (g * u).sum(1, keepdim=True))
        if c["scores"] == "sigmoid":
            d = d * (1.0 - picked)
        dl.scatter_add_(1, ids, d)
    elif c["scores"] == "sigmoid":
        dl.scatter_add_(1, ids, g * u * (1.0 - u))
    else:
        dl.scatter_add_(1, ids, g)
        dl = torch.where(out, torch.zeros_like(dl), score * (dl - (g * u).sum(1, keepdim=True)))
    return {**result, "dlogits": dl.to(logits.dtype)}


def _plain_combine(s):
    c = s["case"]
    y = s["y"].float().unflatten(0, (c["tokens"], c["k"]))
    w = s["weights"]
    out = (y * w[:, :, None]).sum(1).to(s["y"].dtype)
    if c["op"] == "combine":
        return out
    d = s["dout"].float()
    return {"out": out, "dy": (d[:, None, :] * w[:, :, None]).flatten(0, 1).to(s["y"].dtype),
            "dweights": (y * d[:, None, :]).sum(2)}


def _power(top):
    """The least exponent with top <= 448 * 2^exponent, not below -126."""
    m, e = torch.frexp(top)
    e = e - 9 + (m > 0.875).to(e.dtype)
    return torch.where(top > 0, e.clamp_min(-126), torch.full_like(e, -126))


def _eight(v, e):
    return torch.ldexp(v, -e).clamp(-MOST, MOST).to(torch.float8_e4m3fn).float()


def _rows_eight(v):
    """The float32 values of rows taken to 8 bits."""
    h = v.shape[1]
    b = _padded(v.float(), -1).unflatten(1, (-1, BLOCK))
    e = _power(b.abs().amax(2, keepdim=True))
    return torch.ldexp(_eight(b, e), e).flatten(1)[:, :h]


def _weight_eight(W):
    """The float32 values of a weight taken to 8 bits, and its scales."""
    E, N, K = W.shape
    b = _padded(W.float(), -2, -1).unflatten(2, (-1, BLOCK)).unflatten(1, (-1, BLOCK))
    e = _power(b.abs().amax((2, 4), keepdim=True))
    values = torch.ldexp(_eight(b, e), e).flatten(3, 4).flatten(1, 2)[:, :N, :K]
    return values, torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)[:, :, 0, :, 0]


def _weight_values(codes, scales):
    E, N, K = codes.shape
    s = scales.repeat_interleave(BLOCK, 1)[:, :N].repeat_interleave(BLOCK, 2)[:, :, :K]
    return codes.float() * s


def _lay(ids):
    """Rows sorted by expert, and where each stands when every met expert has a block of equal
    length: (rows, experts met, block of each row, place in it, length)."""
    rows = torch.nonzero(ids >= 0).flatten()
    rows = rows[torch.argsort(ids[rows], stable=True)]
    met, block, count = torch.unique_consecutive(ids[rows].long(), return_inverse=True, return_counts=True)
    place = torch.arange(rows.numel(), device=ids.device) - (torch.cumsum(count, 0) - count)[block]
    return rows, met, block, place, int(count.max()) if count.numel() else 0


def _by_expert(v, ids, weights, n_out, top_k, dtype):
    """out[i] = v[i // top_k] @ weights(experts)[ids[i]], rows of no expert zero."""
    if ids is None:
        return torch.matmul(v, weights(slice(0, 1))[0]).to(dtype)
    rows, met, block, place, length = _lay(ids)
    out = torch.zeros(ids.numel(), n_out, dtype=dtype, device=v.device)
    if rows.numel():
        laid = torch.zeros(met.numel(), length, v.shape[1], device=v.device)
        laid[block, place] = v[rows // top_k]
        out[rows] = torch.bmm(laid, weights(met))[block, place].to(dtype)
    return out


def _plain_product(s):
    c = s["case"]
    t, k = TYPES[c["dtype"]], c["top_k"]
    if c["op"] == "quantize":
        values, scales = _weight_eight(s["W"])
        return {"values": values.to(t), "scales": scales}
    x = _rows_eight(s["x"])
    if c["op"] == "fp8":
        return _by_expert(x, s["ids"], lambda e: _weight_values(s["codes"][e], s["scales"][e]).transpose(1, 2),
                          c["h_out"], k, t)
    W, _ = _weight_eight(s["W"])
    return {"y": _by_expert(x, s["ids"], lambda e: W[e].transpose(1, 2), c["h_out"], k, t),
            "dx": _by_expert(_rows_eight(s["dy"]), s["ids"], lambda e: W[e], c["h_in"], 1, t)}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        plain = _plain_route if op.startswith("route") else _plain_combine if op.startswith("combine") else _plain_product
        return plain(s)
    import adapter_gemv_amd as sgmv
    if op.startswith("route"):
        routes = sgmv.route(s["logits"], c["k"], bias=s["bias"], scores=c["scores"], expert_groups=c["groups"],
                            keep_groups=c["keep"], group_best=c["best"], normalize=c["normalize"], scale=c["scale"])
        result = {"ids": routes.ids, "weights": routes.weights}
        if op == "route_train":
            result["dlogits"] = sgmv.route_backward(torch.empty_like(s["logits"]), s["dweights"], s["logits"], routes)
        return result
    if op.startswith("combine"):
        y, w = s["y"], s["weights"]
        out = sgmv.combine_rows(y.new_empty(c["tokens"], c["h"]), y, w)
        if op == "combine":
            return out
        dy, dw = torch.empty_like(y), torch.empty_like(w)
        sgmv.combine_rows_backward(dy, dw, s["dout"], y, w)
        return {"out": out, "dy": dy, "dweights": dw}
    if op == "quantize":
        q = sgmv.fp8_quantize_weight(s["W"])
        return {"values": sgmv.fp8_dequantize(torch.empty_like(s["W"]), q), "scales": q.scales}
    x, n = s["x"], c["tokens"] * c["top_k"]
    groups = None if s["ids"] is None else sgmv.group_rows(s["ids"], c["experts"])
    if op == "fp8":
        return sgmv.fp8_matmul(x.new_empty(n, c["h_out"]), x, sgmv.Fp8Weight(s["codes"], s["scales"]), groups)
    W = sgmv.fp8_quantize_weight(s["W"] if groups is not None else s["W"][0])
    return {"y": sgmv.fp8_matmul(x.new_empty(n, c["h_out"]), x, W, groups),
            "dx": sgmv.fp8_matmul_dx(x.new_empty(n, c["h_in"]), s["dy"], W, groups)}


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------
def _exact_route(s):
    c = s["case"]
    l = s["logits"].double().cpu().numpy()
    T, E = l.shape
    k, G = c["k"], c["groups"]
    with np.errstate(all="ignore"):
        if c["scores"] == "sigmoid":
            p = 1.0 / (1.0 + np.exp(-l))
        else:
            p = np.exp(l - np.max(l, 1, keepdims=True))
            p /= np.sum(p, 1, keepdims=True)
    b = 0.0 if s["bias"] is None else s["bias"].double().cpu().numpy()
    v = np.where(np.isneginf(l), -np.inf, p + b)
    if c["keep"] < G:
        top = -np.sort(-v.reshape(T, G, E // G), 2)[:, :, : c["best"]]
        total = np.where(np.isneginf(top[:, :, 0]), -np.inf, np.where(np.isneginf(top), 0.0, top).sum(2))
        place = np.argsort(np.argsort(-total, 1, kind="stable"), 1, kind="stable")
        v = np.where(np.repeat(place < c["keep"], E // G, 1), v, -np.inf)
    ids = np.argsort(-v, 1, kind="stable")[:, :k]
    at = np.arange(T)[:, None]
    gone = np.isneginf(v[at, ids])
    q = np.where(gone, 0.0, p[at, ids])
    with np.errstate(all="ignore"):
        u = q / q.sum(1, keepdims=True) if c["normalize"] else q
    u = np.where(gone, 0.0, u)
    result = {"ids": np.where(gone, -1, ids).astype(np.int32), "weights": u * c["scale"]}
    if c["op"] == "route_train":
        g = np.where(gone, 0.0, s["dweights"].double().cpu().numpy() * c["scale"])
        d = np.zeros((T, E))
        if c["normalize"]:
            # du_j / dq_m = (delta_jm - u_j) / total, dq_m / dl_m = q_m (times 1 - q_m)
            inner = u * (g - np.sum(g * u, 1, keepdims=True))
            d[at, ids] += np.where(gone, 0.0, inner * ((1.0 - q) if c["scores"] == "sigmoid" else 1.0))
        elif c["scores"] == "sigmoid":
            d[at, ids] += g * q * (1.0 - q)
        else:
            full = np.zeros((T, E))
            full[at, ids] += g
            safe = np.where(np.isneginf(l), 0.0, p)
            d = safe * (full - np.sum(safe * full, 1, keepdims=True))
        result["dlogits"] = d
    return {name: torch.from_numpy(np.ascontiguousarray(a)).cuda() for name, a in result.items()}


def _exact_combine(s):
    c = s["case"]
    T, k = c["tokens"], c["k"]
    out = torch.zeros(T, c["h"], dtype=torch.float64, device="cuda")
    dy = torch.zeros(T, k, c["h"], dtype=torch.float64, device="cuda") if c["op"] == "combine_train" else None
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        y, w = s["y"][j::k].double(), s["weights"][:, j: j + 1].double()
        out += w * y
        if dy is not None:
            dy[:, j] = w * s["dout"].double()
            dw[:, j] = torch.linalg.vecdot(y, s["dout"].double())
    return out if dy is None else {"out": out, "dy": dy.reshape(T * k, c["h"]), "dweights": dw}


def _exact_eight(v, unit):
    """v in 64 bits, to the nearest 8-bit value times unit."""
    a = v / unit
    step = torch.exp2((torch.frexp(a.abs().clamp_min(2.0 ** -6)).exponent - 1).double() - 3)
    return (torch.round(a / step) * step).clamp(-MOST, MOST) * unit


def _exact_unit(top):
    """The least power of two whose 448-fold is not below top, at least 2^-126."""
    u = torch.full_like(top, 2.0 ** -126)
    guess = torch.exp2(torch.floor(torch.log2(top.clamp_min(2.0 ** -200))) - 10).clamp_min(2.0 ** -126)
    for _ in range(5):
        guess = torch.where(guess * MOST < top, guess * 2, guess)
    return torch.where(top > 0, guess, u)


def _exact_rows(v):
    out = torch.empty(v.shape, dtype=torch.float64, device=v.device)
    for lo in range(0, v.shape[1], BLOCK):
        b = v[:, lo: lo + BLOCK].double()
        out[:, lo: lo + BLOCK] = _exact_eight(b, _exact_unit(b.abs().amax(1, keepdim=True)))
    return out


def _exact_weight(W):
    """One group's weight [h_out, h_in] in 64 bits, taken to 8 bits; and its scales."""
    N, K = W.shape
    top = torch.zeros(-(-N // BLOCK), -(-K // BLOCK), dtype=torch.float64, device=W.device)
    for i in range(top.shape[0]):
        band = W[i * BLOCK: (i + 1) * BLOCK].abs().amax(0).double()
        band = torch.cat([band, band.new_zeros(-K % BLOCK)])
        top[i] = band.reshape(-1, BLOCK).amax(1)
    unit = _exact_unit(top)
    return _exact_eight(W.double(), _spread(unit, N, K)), unit


def _spread(per_block, N, K):
    rows = torch.arange(N, device=per_block.device) // BLOCK
    cols = torch.arange(K, device=per_block.device) // BLOCK
    return per_block[rows][:, cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("route"):
        return _exact_route(s)
    if op.startswith("combine"):
        return _exact_combine(s)
    E, N, K = case["experts"], case["h_out"], case["h_in"]
    if op == "quantize":
        parts = [_exact_weight(W) for W in s["W"]]
        return {"values": torch.stack([p[0] for p in parts]), "scales": torch.stack([p[1] for p in parts])}
    n, k = case["tokens"] * case["top_k"], case["top_k"]
    ids = s["ids"] if s["ids"] is not None else torch.zeros(n, dtype=torch.int32, device="cuda")
    x = _exact_rows(s["x"])
    y = torch.zeros(n, N, dtype=torch.float64, device="cuda")
    if op == "fp8_train":
        dy = _exact_rows(s["dy"])
        dx = torch.zeros(n, K, dtype=torch.float64, device="cuda")
    for e in range(E):
        mine = torch.nonzero(ids == e).flatten()
        if mine.numel() == 0:
            continue
        if op == "fp8":
            w = s["codes"][e].to(torch.float64) * _spread(s["scales"][e].double(), N, K)
        else:
            w = _exact_weight(s["W"][e])[0]
            dx[mine] = dy[mine] @ w
        y[mine] = x[mine // k] @ w.t()
    return y if op == "fp8" else {"y": y, "dx": dx}


if __name__ == "__main__":
    for shown in listed() + [draw(random.Random(i)) for i in range(12)]:
        print(shown, work(shown))
