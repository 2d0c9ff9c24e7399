"""Routing to experts and its gradient against the fp64 oracle.

Ids are compared for equality.  Tolerances, u = 2^-24: a score comes from the exponential of a
float32 difference d of logits (relative error (2 |d| + 4) u with its argument's roundings), sums over
at most 1024 experts in a tree under runs of 16 (at most 30 roundings), and a handful of products and
quotients: (2 |d| + 60) u in all; gradients take that of every term that they sum, and the output
type's rounding once."""
import math

import numpy as np
import pytest

from oracle import routing_oracle as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def types(torch):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def near(got, ref, tol, what):
    """Equal where the reference is not finite, within tol elsewhere."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    ok = ~np.isnan(ref)
    err = np.abs(got - ref)[ok]
    tol = np.broadcast_to(tol, ref.shape)[ok]
    print(f"{what}: worst err/tol {(err / tol).max() if err.size else 0:.3f}", flush=True)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} outside"


def distance(l, scores):
    """How far the exponents of the finite logits are from where they start, [T, E]."""
    f = np.where(np.isfinite(l), l, 0.0)
    if scores == "softmax":
        return np.abs(f - np.where(np.isfinite(l), l, -1e30).max(1, keepdims=True)) * np.isfinite(l)
    return 2 * np.abs(f)


def check(torch, logits, k, what, bias=None, scores="softmax", groups=1, keep=None, best=2, normalize=True,
          scale=1.0, seed=0):
    """Forward and backward of one case; returns the routes."""
    import adapter_gemv_amd as sgmv
    T, E = logits.shape
    routes = sgmv.route(logits, k, bias=bias, scores=scores, expert_groups=groups, keep_groups=keep,
                        group_best=best, normalize=normalize, scale=scale)
    l = logits.double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    ids, w = R.route(l, k, b, scores, groups, keep, best, normalize, scale)
    got = routes.ids.cpu().numpy()
    wrong = np.flatnonzero((got != ids).any(1))
    assert wrong.size == 0, f"{what}: row {wrong[0]}: {got[wrong[0]]} for {ids[wrong[0]]}"
    d = distance(l, scores)
    at = np.where(ids < 0, 0, ids)
    far = np.take_along_axis(d, at, 1)
    far = far + (np.where(ids < 0, 0, far).max(1, keepdims=True) if normalize else 0)
    near(routes.weights.cpu().numpy(), w, np.abs(np.nan_to_num(w)) * (2 * far + 60) * U + 2.0 ** -140, what)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    g = torch.randn(T, k, generator=gen, device="cuda")
    dl = sgmv.route_backward(torch.full_like(logits, float("nan")), g, logits, routes)
    ref, mag = R.route_backward(l, ids, g.double().cpu().numpy(), scores, normalize, scale)
    u, sub = {torch.float32: (U, 2.0 ** -149), torch.float16: (2.0 ** -11, 2.0 ** -25),
              torch.bfloat16: (2.0 ** -8, 2.0 ** -134)}[logits.dtype]
    widest = np.where(ids < 0, 0, far).max(1, keepdims=True)   # of the terms that are summed
    near(dl.double().cpu().numpy(), ref,
         np.abs(np.nan_to_num(ref)) * u + sub + np.nan_to_num(mag) * (4 * widest + 2 * d + 200) * U + 2.0 ** -140,
         what + " backward")
    return routes


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 16, 3), (33, 60, 4), (65, 64, 8), (129, 100, 6), (40, 128, 8),
         (50, 160, 6), (70, 256, 8), (9, 257, 12), (20, 512, 10), (6, 700, 64), (5, 1000, 33), (4, 1024, 64)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_sizes(torch, size, scores, dtype):
    T, E, k = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + E)
    for normalize in (True, False):
        for with_bias in (True, False):
            logits = (torch.randn(T, E, generator=gen, device="cuda") * 2).to(types(torch)[dtype])
            bias = torch.randn(E, generator=gen, device="cuda") * 0.2 if with_bias else None
            check(torch, logits, k, f"{size} {scores} {dtype} {normalize} {with_bias}", bias, scores,
                  normalize=normalize, scale=1.0 if normalize else 2.5)


@pytest.mark.parametrize("groups", [(16, 2, 1, 1, 3), (16, 16, 3, 2, 3), (60, 4, 2, 2, 6), (64, 8, 8, 2, 8),
                                    (96, 3, 1, 1, 32), (128, 16, 4, 2, 8), (256, 8, 4, 2, 8), (256, 32, 5, 1, 9),
                                    (250, 10, 3, 2, 7), (512, 64, 9, 2, 12), (1024, 2, 1, 2, 16), (960, 64, 64, 1, 5),
                                    (1008, 63, 20, 2, 20), (256, 1, 1, 1, 8)],
                         ids=lambda g: "-".join(map(str, g)))
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_expert_groups(torch, groups, scores):
    E, n, keep, best, k = groups
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E + n)
    for dtype in ("f32", "bf16"):
        for with_bias in (True, False):
            logits = (torch.randn(45, E, generator=gen, device="cuda") * 1.5).to(types(torch)[dtype])
            bias = torch.randn(E, generator=gen, device="cuda") * 0.1 if with_bias else None
            check(torch, logits, k, f"{groups} {scores} {dtype} {with_bias}", bias, scores, n, keep, best, scale=2.5)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep", [(16, 1, 1), (60, 4, 2), (256, 8, 4), (1024, 16, 5)])
def test_ties_go_to_the_lowest(torch, scores, E, groups, keep):
    """Few different logits, zeros of both signs, a bias of zeros and one that repeats."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E)
    for dtype in ("f32", "f16", "bf16"):
        for bias in (None, torch.zeros(E, device="cuda"), (torch.arange(E, device="cuda") % 3).float() * 0.125):
            logits = torch.randint(-2, 3, (60, E), generator=gen, device="cuda").to(types(torch)[dtype]) * 0.5
            logits = torch.where(torch.rand(60, E, generator=gen, device="cuda") < 0.2, -0.0 * logits.abs(), logits)
            logits[0] = 0.25
            for best in (1, 2):
                check(torch, logits, min(12, E), f"{scores} {dtype} best {best}", bias, scores, groups, keep, best)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_values_next_to_each_other(torch, scores):
    """Values that choose and that float32 does not tell apart: logits one step from each other, and
    biases that undo a difference of scores up to a few parts in 2^30."""
    E = 64
    base = torch.full((40, E), 0.7, device="cuda")
    step = torch.arange(E, device="cuda", dtype=torch.float32)
    logits = base + (step * 17 % 64) * 2.0 ** -24 * torch.linspace(1, 4, 40, device="cuda")[:, None]
    check(torch, logits, 8, f"{scores} steps", torch.zeros(E, device="cuda"), scores)
    check(torch, logits, 8, f"{scores} steps, groups", None, scores, 8, 3, 2)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    l = torch.randn(1, E, generator=gen, device="cuda")
    s = torch.tensor(R.scores_of(l[0].double().tolist(), scores), dtype=torch.float64, device="cuda")
    bias = (1.0 - s).float()      # s + bias = 1 up to float32's rounding of the bias
    check(torch, l.repeat(3, 1), 9, f"{scores} biases", bias, scores)
    check(torch, l.repeat(3, 1), 9, f"{scores} biases, groups", bias, scores, 8, 3, 2)
    check(torch, l.repeat(3, 1), 9, f"{scores} biases, best of a group", bias, scores, 8, 3, 1)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,keep", [(32, 5, 1, 1), (256, 8, 1, 1), (250, 15, 1, 1), (256, 16, 1, 1),
                                             (512, 20, 1, 1), (1024, 64, 1, 1), (64, 6, 8, 3), (256, 8, 8, 4),
                                             (256, 9, 32, 5), (512, 30, 16, 7)])
def test_pairs_that_float32_leaves_open(torch, scores, E, k, groups, keep):
    """Values far from each other but for pairs a step apart or equal: inside the choice, across its end,
    and among the sums of groups, of which each two hold the same values up to a step."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E + k)
    T, half = 96, E // 2

    def order(*shape):
        return torch.rand(*shape, generator=gen, device="cuda").argsort(-1)

    a = order(T, half).float() * (3.0 / half) - 1.5
    up = torch.nextafter(a, torch.full_like(a, 9.0))
    b = torch.where(torch.rand(T, half, generator=gen, device="cuda") < 0.5, a, up)
    if groups == 1:
        logits = torch.cat([a, b], 1).gather(1, order(T, E))
    else:
        per = E // groups
        pairs = torch.stack([a.view(T, groups // 2, per), b.view(T, groups // 2, per)], 2)
        logits = pairs.view(T, groups, per).gather(2, order(T, groups, per)).view(T, E)
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.375, device="cuda")):
        for best in (1, 2):
            check(torch, logits, k, f"{E} {k} {scores} best {best}", bias, scores, groups, keep, best)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,groups,keep", [(9, 4, 3, 2), (64, 8, 1, 1), (256, 8, 8, 4), (1024, 20, 4, 1)])
@pytest.mark.parametrize("normalize", [True, False])
def test_masks(torch, scores, E, k, groups, keep, normalize):
    """Masks by minus infinity down to nothing, masks by the type's lowest value, biases of minus and
    plus infinity."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E)
    for dtype in ("f32", "f16", "bf16"):
        t = types(torch)[dtype]
        logits = torch.randn(40, E, generator=gen, device="cuda").to(t)
        gone = torch.rand(40, E, generator=gen, device="cuda") < torch.linspace(0, 1, 40, device="cuda")[:, None]
        gone[30:] = True
        gone[31, E - 1] = False
        gone[32, :2] = False
        bias = torch.randn(E, generator=gen, device="cuda") * 0.1
        for b in (None, bias):
            hard = torch.where(gone, torch.full_like(logits, -math.inf), logits)
            r = check(torch, hard, k, f"{scores} {dtype} masked", b, scores, groups, keep, normalize=normalize)
            assert bool((r.ids[30] == -1).all()) and not bool(r.weights[30].any())
            low = torch.where(gone, torch.full_like(logits, torch.finfo(t).min), logits)
            check(torch, low, k, f"{scores} {dtype} lowest", b, scores, groups, keep, normalize=normalize)
        bias[1::3] = -math.inf
        bias[2] = math.inf
        check(torch, logits, k, f"{scores} {dtype} infinite biases", bias, scores, groups, keep, normalize=normalize)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_far_logits(torch, scores, normalize):
    """Logits up to the end of the type, all of them small as well: scores below what float32 holds."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    for shift, spread in ((0.0, 30.0), (-60.0, 3.0), (-90.0, 3.0), (-300.0, 50.0), (80.0, 30.0), (-6e4, 10.0)):
        logits = torch.randn(20, 40, generator=gen, device="cuda") * spread + shift
        check(torch, logits, 5, f"{scores} {shift} {spread}", None, scores, normalize=normalize)
    big = torch.randn(6, 40, generator=gen, device="cuda") * 1e38
    check(torch, big, 5, f"{scores} 1e38", None, scores, normalize=normalize)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("groups,keep,best", [(1, 1, 1), (4, 2, 2), (4, 2, 1)])
def test_what_is_no_number(torch, scores, normalize, groups, keep, best):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    for dtype in ("f32", "f16"):
        for bias in (None, torch.randn(24, generator=gen, device="cuda") * 0.1):
            logits = torch.randn(12, 24, generator=gen, device="cuda").to(types(torch)[dtype])
            logits[1, 7] = math.nan
            logits[2, 23] = math.inf
            logits[3] = math.nan
            logits[4, ::2], logits[4, 5] = -math.inf, math.nan
            logits[5, [2, 9]] = math.inf
            logits[6, 3], logits[6, 4] = -math.nan, math.nan
            check(torch, logits, 5, f"{scores} {dtype}", bias, scores, groups, keep, best, normalize=normalize)
    bias = torch.zeros(24, device="cuda")
    bias[11] = math.nan
    check(torch, torch.randn(5, 24, device="cuda", generator=gen), 5, "bias", bias, scores, groups, keep, best,
          normalize=normalize)


def test_strides_streams_and_nothing(torch):
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    for dtype in ("f32", "f16", "bf16"):
        for E, wide, at in ((60, 64, 0), (60, 61, 1), (256, 300, 7), (256, 264, 8), (8, 8, 0), (128, 129, 0)):
            store = torch.full((37, wide), float("nan"), device="cuda", dtype=types(torch)[dtype])
            logits = store[:, at:at + E]
            if at + E > wide:
                continue
            logits.copy_(torch.randn(37, E, generator=gen, device="cuda"))
            r = check(torch, logits, 6, f"{dtype} {E} {wide} {at}")
            out = torch.full((37, wide + 3), 7.0, device="cuda", dtype=types(torch)[dtype])
            g = torch.randn(37, 6, generator=gen, device="cuda")
            sgmv.route_backward(out[:, 1:1 + E], g, logits, r)
            same = sgmv.route_backward(torch.empty(37, E, device="cuda", dtype=out.dtype), g, logits, r)
            assert torch.equal(out[:, 1:1 + E], same) and bool((out[:, 0] == 7).all()) and bool((out[:, 1 + E:] == 7).all())
    none = sgmv.route(torch.empty(0, 16, device="cuda"), 4)
    assert tuple(none.ids.shape) == (0, 4) and tuple(none.weights.shape) == (0, 4)
    sgmv.route_backward(torch.empty(0, 16, device="cuda"), torch.empty(0, 4, device="cuda"), torch.empty(0, 16, device="cuda"), none)
    stream = torch.cuda.Stream()
    logits = torch.randn(500, 128, generator=gen, device="cuda")
    torch.cuda.synchronize()
    a = sgmv.route(logits, 8, scores="sigmoid", stream=stream)
    stream.synchronize()
    b = sgmv.route(logits, 8, scores="sigmoid")
    assert torch.equal(a.ids, b.ids) and torch.equal(a.weights, b.weights)
    # one row of any stride
    row = torch.randn(4, 64, generator=gen, device="cuda")[1:2]
    check(torch, row.as_strided((1, 64), (3, 1), 64), 4, "one row")


def test_many_rows(torch):
    """More rows than a launch has workgroups at once, each against its own."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    for E, k, dtype in ((4, 2, "f16"), (64, 6, "bf16"), (256, 8, "f32")):
        T = 70001
        some = torch.randn(997, E, generator=gen, device="cuda").to(types(torch)[dtype])
        at = torch.arange(T, device="cuda") % 997
        all_of = sgmv.route(some[at], k, scores="sigmoid")
        few = check(torch, some[:50], k, f"{E}", None, "sigmoid")
        once = sgmv.route(some, k, scores="sigmoid")
        assert torch.equal(all_of.ids, once.ids[at]) and torch.equal(all_of.weights, once.weights[at])
        assert torch.equal(once.ids[:50], few.ids)
        g = torch.randn(997, k, generator=gen, device="cuda")
        d = sgmv.route_backward(torch.empty(T, E, device="cuda", dtype=some.dtype), g[at].contiguous(), some[at], all_of)
        d1 = sgmv.route_backward(torch.empty_like(some), g, some, once)
        assert torch.equal(d, d1[at])


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_backward_of_any_ids(torch, scores, normalize):
    """Ids that no call of route made: an expert twice, places without one, numbers out of range."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    for E, k in ((12, 5), (200, 64)):
        logits = torch.randn(30, E, generator=gen, device="cuda")
        logits[4, ::3] = -math.inf
        ids = torch.randint(-2, E + 2, (30, k), generator=gen, device="cuda", dtype=torch.int32)
        ids[0] = 3
        ids[1] = -1
        ids[2, :] = torch.iinfo(torch.int32).max
        g = torch.randn(30, k, generator=gen, device="cuda")
        routes = sgmv.Routes(ids, torch.empty(30, k, device="cuda"), scores, normalize, 1.5)
        runs = [sgmv.route_backward(torch.empty_like(logits), g, logits, routes) for _ in range(3)]
        assert torch.equal(runs[0], runs[1]) and torch.equal(runs[0], runs[2])
        l = logits.double().cpu().numpy()
        ref, mag = R.route_backward(l, ids.cpu().numpy(), g.double().cpu().numpy(), scores, normalize, 1.5)
        near(runs[0].cpu().numpy(), ref, np.abs(ref) * U + mag * (6 * distance(l, scores).max() + 200) * U + 2.0 ** -140,
             f"{scores} {E}")


def test_gradient_against_differences(torch):
    """Of the call itself: weights in float32, steps of 2^-6 in a smooth place (third differences are below 1: an
    error of 2^-12 of the step's quotient, and 2 * 2^-23 / 2^-6 from rounding)."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    for scores in ("softmax", "sigmoid"):
        for normalize in (True, False):
            l = torch.linspace(-1, 1, 10, device="cuda")[torch.randperm(10, generator=gen, device="cuda")][None]
            g = torch.randn(1, 3, generator=gen, device="cuda")
            r = sgmv.route(l, 3, scores=scores, normalize=normalize)
            d = sgmv.route_backward(torch.empty_like(l), g, l, r)
            h = 2.0 ** -6
            for i in range(10):
                f = []
                for s in (h, -h):
                    x = l.clone()
                    x[0, i] += s
                    q = sgmv.route(x, 3, scores=scores, normalize=normalize)
                    assert torch.equal(q.ids.sort().values, r.ids.sort().values)
                    f.append(sum(float(q.weights[0, j]) * float(g[0, (r.ids[0] == q.ids[0, j]).nonzero()[0, 0]])
                                 for j in range(3)))
                assert abs((f[0] - f[1]) / (2 * h) - float(d[0, i])) < 3 * float(g.abs().max()) * (2.0 ** -12 + 2.0 ** -16)


CUTS = [(4, 2, 1, 1), (8, 4, 1, 2), (64, 32, 7, 3), (256, 8, 3, 8), (128, 16, 5, 17), (512, 8, 3, 8), (1024, 64, 9, 12)]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [100.0, 1e4, 1e6])
@pytest.mark.parametrize("E,groups,keep,k", CUTS)
def test_biases_that_cancel_in_a_group(torch, scores, size, E, groups, keep, k):
    """A group's two best have biases of opposite sign, whose sum says nothing about what float32 rounded off them;
    another group without biases has nearly the same sum, and the cut runs between two such groups."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E + groups)
    T, per, half = 200, E // groups, groups // 2
    logits = torch.full((T, half, 2, per), -30.0, device="cuda")
    bias = torch.zeros(half, 2, per, device="cuda")
    logits[..., :2] = torch.randn(T, half, 1, 2, generator=gen, device="cuda")
    apart = min(1.0, size * 2.0 ** -23 * (5 if scores == "sigmoid" else 2 * groups))
    logits[:, :, 1, 1] += apart * torch.randn(T, half, generator=gen, device="cuda")
    bias[:, 0] = -3 * size
    bias[:, 0, 0], bias[:, 0, 1] = size, -size
    at = torch.rand(groups, generator=gen, device="cuda").argsort()
    logits, bias = logits.view(T, groups, per)[:, at].reshape(T, E), bias.view(groups, per)[at].reshape(E)
    check(torch, logits, k, f"{scores} {size} {E} in {groups}", bias, scores, groups, keep, 2)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("E,groups,keep,k", CUTS)
def test_biases_of_the_largest_size(torch, scores, best, E, groups, keep, k):
    """The largest finite biases of both signs on none, some and all experts of a group (masks by the type's lowest
    value among them), beside groups without an expert: sums past float32's range."""
    most = torch.finfo(torch.float32).max
    gen = torch.Generator(device="cuda")
    gen.manual_seed(E + best)
    T, per = 60, E // groups
    kinds = torch.tensor([most, -most, 0.6 * most, -0.6 * most], device="cuda")
    for sides in (2, 4):
        for share in (0.3, 0.7, 1.0):
            logits = torch.randn(T, groups, per, generator=gen, device="cuda")
            logits[torch.rand(T, groups, generator=gen, device="cuda") < 0.4] = -math.inf
            at = torch.randint(0, sides, (groups, 1), generator=gen, device="cuda").expand(-1, per).clone()
            mixed = torch.rand(groups, per, generator=gen, device="cuda") < 0.2
            at[mixed] = torch.randint(0, sides, (groups, per), generator=gen, device="cuda")[mixed]
            large = torch.rand(groups, per, generator=gen, device="cuda") < share
            bias = torch.where(large, kinds[at], torch.randn(groups, per, generator=gen, device="cuda") * 0.1)
            check(torch, logits.view(T, E), k, f"{scores} {E} in {groups}, {sides} {share}", bias.view(E), scores, groups,
                  keep, best)
    # every expert masked but those of groups that are not there
    logits = torch.randn(T, groups, per, generator=gen, device="cuda")
    logits[:, ::2] = -math.inf
    bias = torch.full((groups, per), -most, device="cuda")
    bias[::2] = 0.0
    r = check(torch, logits.view(T, E), min(k, keep * per), f"{scores} {E} in {groups}, lowest", bias.view(E), scores,
              groups, keep, best)
    assert bool((r.ids[:, 0] >= 0).all())
