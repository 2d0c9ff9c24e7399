"""The products of expert layers and of 4-bit weights: cases, plain forms and 64-bit values.

A case names one pass through one operator:

* ``forward``   rows grouped by expert, each row times its own expert's weight,
                ``y[i] = x[i // top_k] @ W[ids[i]].T``;
* ``backward``  the two gradients of that product, ``dx[i] = dy[i] @ W[ids[i]]`` (one for each
                row, also where several rows share an x) and ``dW[e] = sum_i dy[i].T x[i // top_k]``
                over the rows of expert e;
* ``quantize``  16-bit values to microscaled 4-bit floating point (blocks of 32 along a row, one
                power of two each, elements of two exponent bits and one mantissa bit) and back;
* ``mx``        16-bit rows times weights held in that format, dense or by expert;
* ``mx_both``   the same with the rows taken to that format too, inside the call.

Rows whose id is negative belong to no expert here (another device holds it, or the row is
padding): their output rows are zero and they add nothing to any gradient.
"""
import math
import random

import torch

own = False

BF16, F16 = "bf16", "f16"
BLOCK = 32


# --------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------
def _rows(op, name, dtype, tokens, top_k, experts, h_in, h_out, skew=0.0, away=0.0):
    return {"name": name, "op": op, "dtype": dtype, "tokens": tokens, "top_k": top_k,
            "experts": experts, "h_in": h_in, "h_out": h_out, "skew": skew, "away": away}


def listed():
    return [
        # one generated token in a small expert layer: two experts' weights, latency
        _rows("forward", "experts_one_token", BF16, 1, 2, 8, 4096, 1024),
        # a decode batch over many narrow experts: about half of them are met, few rows each
        _rows("forward", "experts_decode", F16, 32, 2, 64, 4096, 1024, 0.3),
        # a prompt of odd length through wide experts, some popular
        _rows("forward", "experts_prompt", BF16, 1531, 2, 8, 5120, 13824, 0.6),
        # many prompts together over narrow experts, a tenth of the rows held elsewhere
        _rows("forward", "experts_many_prompts", F16, 8192, 4, 64, 4096, 1024, 0.3, 0.1),
        # a small training step: odd sizes, ragged
        _rows("backward", "experts_train_small", F16, 777, 1, 4, 1032, 520, 0.6),
        # a training step of full width
        _rows("backward", "experts_train", BF16, 8192, 2, 16, 4096, 4096, 0.3),
        # a prompt's activations, written in 4 bits (as a cache or a checkpoint would hold them)
        {"name": "quantize_activations", "op": "quantize", "dtype": BF16, "rows": 2048, "h": 5120},
        # a feed-forward weight, once when it is loaded
        {"name": "quantize_weight", "op": "quantize", "dtype": F16, "rows": 28672, "h": 8192},
        # one generated token through a dense projection held in 4 bits
        _rows("mx", "mx_one_token", BF16, 1, 1, 1, 4096, 4096),
        # a decode batch through experts held in 4 bits
        _rows("mx", "mx_experts_decode", F16, 16, 2, 8, 5120, 13824, 0.3),
        # a prompt through experts held in 4 bits, activations left in 16
        _rows("mx", "mx_experts_prompt", BF16, 1021, 2, 8, 4096, 8192, 0.6),
        # the mixed batch's rows through a wide dense projection, both sides in 4 bits
        _rows("mx_both", "mx_both_prompt", BF16, 2112, 1, 1, 8192, 28672),
    ]


def _log(rng, lo, hi, unit=1):
    return max(unit, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit)) * unit)


def draw(rng):
    top = [work(c) for c in listed()]
    most = {k: max(w[k] for w in top) / 2 for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["forward", "forward", "backward", "quantize", "mx", "mx", "mx_both"])
        dtype = rng.choice([BF16, F16])
        if op == "quantize":
            c = {"op": op, "dtype": dtype, "rows": _log(rng, 1, 30000), "h": _log(rng, 512, 16384, 32)}
        else:
            unit = 32 if op.startswith("mx") else 8
            experts = 1 if op.startswith("mx") and rng.random() < 0.5 else _log(rng, 2, 96)
            c = _rows(op, "", dtype, _log(rng, 64 if op == "backward" else 1, 12000),
                      rng.randint(1, min(4, experts)), experts, _log(rng, 512, 14336, unit),
                      _log(rng, 256, 14336, 8), rng.choice([0.0, 0.3, 0.6, 1.0]),
                      rng.choice([0.0, 0.0, 0.25]) if experts > 1 else 0.0)
            del c["name"]
            if experts * c["h_in"] * c["h_out"] > 6e8:
                continue
        w = work(c)
        if 3 << 10 not in c.values() and w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"]:
            return c


def _popularity(case):
    p = [(e + 1.0) ** -case["skew"] for e in range(case["experts"])]
    return [v / sum(p) for v in p]


def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["h"]
        return {"bytes": 4 * n, "flops": 2 * n}
    n = case["tokens"] * case["top_k"]
    here = n * (1.0 - case["away"])
    met = sum(1.0 - (1.0 - p) ** here for p in _popularity(case))
    weight = case["h_in"] * case["h_out"]
    flops = 2.0 * here * weight
    x, y = 2 * case["tokens"] * case["h_in"], 2 * n * case["h_out"]
    if case["op"] == "backward":
        # x, dy and W are read, dx (for each row) and the whole dW are written
        return {"bytes": x + y + 2 * met * weight + 2 * n * case["h_in"] + 2 * case["experts"] * weight,
                "flops": 2 * flops}
    per = 2.0 if case["op"] == "forward" else 0.5 + 1.0 / BLOCK
    return {"bytes": x + y + per * met * weight, "flops": flops}


# --------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------
def _type(case):
    return torch.bfloat16 if case["dtype"] == BF16 else torch.float16


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
    t = _type(case)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(t)

    if case["op"] == "quantize":
        # rows of different size, a few large columns: what activations and weights look like
        x = torch.randn(case["rows"], case["h"], generator=gen, device="cuda")
        x *= torch.exp(torch.randn(case["rows"], 1, generator=gen, device="cuda"))
        x[:, torch.randperm(case["h"], generator=gen, device="cuda")[: case["h"] // 128 + 1]] *= 20.0
        return {"case": case, "x": x.to(t)}
    E, K, N = case["experts"], case["h_in"], case["h_out"]
    s = {"case": case, "x": normal(case["tokens"], K),
         "W": normal(E, N, K, std=K ** -0.5),
         "ids": _ids(case, gen) if E > 1 else None}
    if case["op"] == "backward":
        s["dy"] = normal(case["tokens"] * case["top_k"], N, std=N ** -0.5)
        if s["ids"] is None:
            s["ids"] = torch.zeros(case["tokens"] * case["top_k"], dtype=torch.int32, device="cuda")
    if case["op"].startswith("mx"):
        s["codes"], s["scales"] = _encode(s.pop("W"))
    return s


# --------------------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------------------
def _encode(v):
    """(codes uint8 [..., h / 2], scales uint8 [..., h / 32]) of v [..., h].  A block's scale is
    2^(floor(log2(largest magnitude)) - 2), stored with bias 127; the element at an even place is
    the low half of its byte; ties go to the even code, what passes 6 becomes 6."""
    b = v.float().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.full_like(top, -127, dtype=torch.int32))
    e = e.clamp(-127, 127)
    a = torch.ldexp(b.abs(), -e)
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75).to(torch.uint8) + (a > 1.25).to(torch.uint8)
            + (a >= 1.75).to(torch.uint8) + (a > 2.5).to(torch.uint8) + (a >= 3.5).to(torch.uint8)
            + (a > 5.0).to(torch.uint8)) + 8 * torch.signbit(b).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], (e + 127).to(torch.uint8).squeeze(-1)


def _decode(codes, scales):
    """The float32 values that 4-bit codes and their scales stand for."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0,
                          -4.0, -6.0], device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    return torch.ldexp(v.unflatten(-1, (-1, BLOCK)), scales.int()[..., None] - 127).flatten(-2)


def _blocks(ids):
    """Rows sorted by expert, and where each stands when every met expert has a block of equal
    length: (rows, experts met, block of each row, place in it, length)."""
    rows = torch.nonzero(ids >= 0).flatten()
    rows = rows[torch.argsort(ids[rows], stable=True)]
    met, block, count = torch.unique_consecutive(ids[rows].long(), return_inverse=True, return_counts=True)
    place = torch.arange(rows.numel(), device=ids.device) - (torch.cumsum(count, 0) - count)[block]
    return rows, met, block, place, int(count.max()) if count.numel() else 0


def _lay(v, at, rows):
    out = torch.zeros(at[1].numel(), at[4], v.shape[1], device=v.device)
    out[at[2], at[3]] = v[rows].float()
    return out


def _plain_product(x, ids, weights, n, n_out, top_k, dtype):
    """y[i] = x[i // top_k] @ W[ids[i]].T; weights(experts) gives those experts' in float32."""
    if ids is None:
        return torch.matmul(x.float(), weights(slice(0, 1))[0].t()).to(dtype)
    at = _blocks(ids)
    y = torch.zeros(n, n_out, dtype=dtype, device=x.device)
    p = torch.bmm(_lay(x, at, at[0] // top_k), weights(at[1]).transpose(1, 2))
    y[at[0]] = p[at[2], at[3]].to(dtype)
    return y


def _plain(s):
    c = s["case"]
    t = _type(c)
    if c["op"] == "quantize":
        return _decode(*_encode(s["x"])).to(t)
    n = c["tokens"] * c["top_k"]
    if c["op"] == "forward":
        return _plain_product(s["x"], s["ids"], lambda e: s["W"][e].float(), n, c["h_out"], c["top_k"], t)
    if c["op"] == "backward":
        at = _blocks(s["ids"])
        dy = _lay(s["dy"], at, at[0])
        dx = torch.zeros(n, c["h_in"], dtype=t, device=dy.device)
        dx[at[0]] = torch.bmm(dy, s["W"][at[1]].float())[at[2], at[3]].to(t)
        dw = torch.zeros(c["experts"], c["h_out"], c["h_in"], dtype=t, device=dy.device)
        dw[at[1]] = torch.bmm(dy.transpose(1, 2), _lay(s["x"], at, at[0] // c["top_k"])).to(t)
        return {"dx": dx, "dw": dw}
    x = s["x"] if c["op"] == "mx" else _decode(*_encode(s["x"]))
    return _plain_product(x, s["ids"], lambda e: _decode(s["codes"][e], s["scales"][e]), n, c["h_out"],
                          c["top_k"], t)


def run(s):
    if not own:
        return _plain(s)
    import adapter_gemv_amd as sgmv
    c, x = s["case"], s["x"]
    if c["op"] == "quantize":
        return sgmv.mx_dequantize(torch.empty_like(x), sgmv.mx_quantize(x))
    groups = None if s["ids"] is None else sgmv.group_rows(s["ids"], c["experts"])
    n = c["tokens"] * c["top_k"]
    if c["op"] == "backward":
        dx = sgmv.group_matmul_dx(x.new_empty(n, c["h_in"]), s["dy"], s["W"], groups)
        dw = sgmv.group_matmul_dw(torch.empty_like(s["W"]), x, s["dy"], groups)
        return {"dx": dx, "dw": dw}
    y = x.new_empty(n, c["h_out"])
    if c["op"] == "forward":
        return sgmv.group_matmul(y, x, s["W"], groups)
    weight = sgmv.MxTensor(s["codes"], s["scales"])
    return sgmv.mx_matmul(y, x if c["op"] == "mx" else sgmv.mx_quantize(x), weight, groups)


# --------------------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------------------
def _exact_round(v):
    """v [..., h] in float64, rounded to the 4-bit format's nearest values."""
    b = v.double().unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    unit = torch.exp2((torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 2).clamp(-127, 127))
    # log2 may round up to a whole number just below a power of two
    unit = torch.where(unit * 4 > top.clamp_min(2.0 ** -140), (unit / 2).clamp_min(2.0 ** -127), unit)
    a = b / unit
    step = torch.where(a.abs() < 2, 0.5, torch.where(a.abs() < 4, 1.0, 2.0)).double()
    return ((torch.round(a / step) * step).clamp(-6, 6) * unit).flatten(-2)


def _exact_weight(codes, scales):
    half = torch.stack((codes % 16, codes // 16), -1).flatten(-2).long()
    e, m = (half % 8) // 2, (half % 2).double()
    size = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
    size = torch.where(half >= 8, -size, size)
    return size * torch.repeat_interleave(torch.exp2(scales.double() - 127), BLOCK, -1)


def exact(case, seed):
    s = prepare(case, seed)
    x = s["x"]
    if case["op"] == "quantize":
        return torch.cat([_exact_round(v) for v in x.split(4096)])
    n, k = case["tokens"] * case["top_k"], case["top_k"]
    ids = s["ids"] if s["ids"] is not None else torch.zeros(n, dtype=torch.int32, device="cuda")
    if case["op"] == "mx_both":
        x = _exact_round(x)
    y = torch.zeros(n, case["h_out"], dtype=torch.float64, device="cuda")
    dx = torch.zeros(n, case["h_in"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(case["experts"], case["h_out"], case["h_in"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        mine = torch.nonzero(ids == e).flatten()
        w = s["W"][e].double() if "W" in s else _exact_weight(s["codes"][e], s["scales"][e])
        if case["op"] == "backward":
            d = s["dy"][mine].double()
            dx[mine] = d @ w
            dw[e] = d.t() @ x[mine // k].double()
        else:
            y[mine] = x[mine // k].double() @ w.t()
    return {"dx": dx, "dw": dw} if case["op"] == "backward" else y


if __name__ == "__main__":
    for shown in listed() + [draw(random.Random(i)) for i in range(12)]:
        print(shown, work(shown))
