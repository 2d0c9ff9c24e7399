"""Products grouped by row ids and their gradients on the GPU, against the fp64 oracle.

Tolerance of an output: its own rounding to 16 bits (half a unit in the last place, u |ref|,
plus half the smallest subnormal) and the float32 sum's, at most (depth + 32) 2^-23 times the
sum of the terms' magnitudes (every partial sum and product rounded or truncated once)."""
import sys

import numpy as np
import pytest

from oracle import grouped_oracle as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


def _dt(torch, dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def tolerance(ref, mag, depth, dtype):
    u, sub = (2.0 ** -8, 2.0 ** -134) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)
    return u * np.abs(ref) + sub + (1 + u) * (depth + 32) * 2.0 ** -23 * mag


def close(got, ref, mag, depth, dtype, what):
    err, tol = np.abs(got - ref), tolerance(ref, mag, depth, dtype)
    say(f"{what}: max|err| {err.max() if err.size else 0:.3e}, "
        f"worst err/tol {(err / tol).max() if err.size else 0:.3f}")
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} outside"


def f64(t):
    return t.double().cpu().numpy()


def padded(torch, rows, cols, dtype, pad, gen, std=1.0, fill=float("nan")):
    """A [rows, cols] view of a buffer with `pad` more columns that hold NaN."""
    buf = torch.full((rows, cols + pad), fill, dtype=dtype, device="cuda")
    buf[:, :cols] = (torch.randn(rows, cols, generator=gen, device="cuda") * std).to(dtype)
    return buf[:, :cols], buf


def problem(torch, seed, dtype, x_rows, share, E, K, N, ids=None, pad=0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _dt(torch, dtype)
    n = x_rows * share
    if ids is None:
        ids = torch.randint(0, E, (n,), generator=gen, device="cuda", dtype=torch.int32)
    else:
        ids = torch.tensor(ids, dtype=torch.int32, device="cuda")
    x, _ = padded(torch, x_rows, K, t, pad, gen)
    dy, _ = padded(torch, n, N, t, pad, gen, N ** -0.5)
    W = (torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5).to(t)
    return x, dy, W, ids


def check_all(torch, x, dy, W, ids, share, dtype, what, pad=0):
    """Forward and both gradients through the public calls, every element."""
    import adapter_gemv_amd as sgmv
    E, N, K = W.shape
    n = len(ids)
    groups = sgmv.group_rows(ids, E)
    ids_h = ids.cpu().numpy()

    def out(rows, cols):
        buf = torch.full((rows, cols + pad), 7.0, dtype=W.dtype, device="cuda")
        return buf[:, :cols], buf

    y, ybuf = out(n, N)
    dx, dxbuf = out(n, K)
    dW = torch.full_like(W, 7.0)
    say(f"{what}: n={n} share={share} E={E} K={K} N={N} {dtype} pad={pad}")
    sgmv.group_matmul(y, x, W, groups)
    sgmv.group_matmul_dx(dx, dy, W, groups)
    sgmv.group_matmul_dw(dW, x, dy, groups)
    torch.cuda.synchronize()
    X, D, Wd = f64(x), f64(dy), f64(W)
    ref, mag = G.group_matmul(X, Wd, ids_h, share)
    close(f64(y), ref, mag, K, dtype, what + " y")
    ref, mag = G.group_matmul_dx(D, Wd, ids_h)
    close(f64(dx), ref, mag, N, dtype, what + " dx")
    ref, mag = G.group_matmul_dw(X, D, ids_h, E, share)
    close(f64(dW), ref, mag, n, dtype, what + " dW")
    if pad:
        assert torch.all(ybuf[:, N:] == 7.0) and torch.all(dxbuf[:, K:] == 7.0), "padding written"


# --------------------------------------------------------------------------------------
# group tables
# --------------------------------------------------------------------------------------
@pytest.mark.parametrize("n,E", [(0, 3), (1, 1), (5, 1), (63, 2), (64, 7), (65, 64), (1000, 65),
                                 (1023, 300), (5000, 512), (5000, 513), (20011, 1024), (40000, 8),
                                 (8191, 3), (8192, 3), (300001, 77)])
def test_group_rows(torch, n, E):
    import adapter_gemv_amd as sgmv
    rng = np.random.default_rng(n + E)
    for kind in ("uniform", "skewed", "outside", "one"):
        if kind == "uniform":
            ids = rng.integers(0, E, n)
        elif kind == "skewed":
            ids = np.minimum(rng.geometric(0.3, n) - 1, E - 1)
        elif kind == "outside":
            ids = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31, 0, E - 1], n)
        else:
            ids = np.full(n, E - 1)
        g = sgmv.group_rows(torch.tensor(ids, dtype=torch.int32, device="cuda"), E)
        starts, perm = G.group_rows(ids, E)
        assert np.array_equal(g.starts.cpu().numpy(), starts), kind
        assert np.array_equal(g.perm.cpu().numpy(), perm), kind


# --------------------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------------------
def spread(got, ref_of, outs, what, dtype, depth):
    """Blocks of rows against the oracle, so that a large result needs little memory."""
    for lo in range(0, outs, 512):
        rows = np.arange(lo, min(outs, lo + 512))
        close(got(rows), *ref_of(rows), depth, dtype, f"{what} rows {lo}..")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,share,E,depth,wide", [(4200, 1, 3, 200, 4096), (2300, 2, 2, 392, 4000),
                                                     (4097, 1, 1, 72, 4104)])
def test_enough_work_for_the_largest_tiles(torch, dtype, rows, share, E, depth, wide):
    """Products that fill the card with 256 x 256 tiles: ragged groups, rows of no group,
    contracted lengths that end inside a stage, an odd and an even number of stages."""
    import adapter_gemv_amd as sgmv
    n = rows * share
    rng = np.random.default_rng(7)
    ids = rng.choice(np.arange(-1, E), n, p=np.r_[0.05, np.full(E, 0.95 / E)])
    groups = sgmv.group_rows(torch.tensor(ids, dtype=torch.int32, device="cuda"), E)
    x, dy, W, _ = problem(torch, 17, dtype, rows, share, E, depth, wide, ids=ids, pad=8)
    y = sgmv.group_matmul(torch.empty(n, wide, dtype=x.dtype, device="cuda"), x, W, groups)
    X, D, Wd = f64(x), f64(dy), f64(W)

    def forward(rows_):
        ref, mag = np.zeros((len(rows_), wide)), np.zeros((len(rows_), wide))
        for g in range(E):
            m = ids[rows_] == g
            a = X[rows_[m] // share]
            ref[m], mag[m] = a @ Wd[g].T, np.abs(a) @ np.abs(Wd[g]).T
        return ref, mag

    spread(lambda r: f64(y[torch.tensor(r, device="cuda")]), forward, n, "y", dtype, depth)
    # dx: the contracted dimension is W's rows, the wide one its columns
    Wt = W.transpose(1, 2).contiguous()
    z = torch.randn(n, depth, device="cuda").to(x.dtype) * depth ** -0.5
    dx = sgmv.group_matmul_dx(torch.empty(n, wide, dtype=x.dtype, device="cuda"), z, Wt, groups)
    Z, Wt64 = f64(z), f64(Wt)

    def backward(rows_):
        ref, mag = np.zeros((len(rows_), wide)), np.zeros((len(rows_), wide))
        for g in range(E):
            m = ids[rows_] == g
            ref[m], mag[m] = Z[rows_[m]] @ Wt64[g], np.abs(Z[rows_[m]]) @ np.abs(Wt64[g])
        return ref, mag

    spread(lambda r: f64(dx[torch.tensor(r, device="cuda")]), backward, n, "dx", dtype, depth)
    # dW of a wide weight from few rows: the first ones
    few = 2 * depth // share * share
    x2, _ = padded(torch, few // share, wide, x.dtype, 8, torch.Generator(device="cuda").manual_seed(3))
    ids2 = rng.integers(-1, E, few)
    g2 = sgmv.group_rows(torch.tensor(ids2, dtype=torch.int32, device="cuda"), E)
    dW = sgmv.group_matmul_dw(torch.empty(E, wide, wide, dtype=x.dtype, device="cuda"), x2, dy[:few], g2)
    X2, D2 = f64(x2), D[:few]
    for g in range(E):
        m = np.flatnonzero(ids2 == g)
        a = X2[m // share]
        spread(lambda r: f64(dW[g, torch.tensor(r, device="cuda")]),
               lambda r: (D2[m][:, r].T @ a, np.abs(D2[m][:, r]).T @ np.abs(a)), wide, f"dW {g}", dtype, few)


SHAPES = [
    # x rows, share, E, K, N
    (1, 1, 1, 8, 8), (1, 2, 4, 64, 32), (1, 4, 64, 1024, 264), (2, 1, 3, 72, 40),
    (7, 3, 5, 520, 136), (16, 1, 1, 256, 512), (17, 1, 2, 1032, 8), (33, 2, 8, 8, 1032),
    (64, 2, 6, 200, 328), (65, 1, 1, 4096, 64), (129, 1, 4, 264, 256), (150, 2, 3, 128, 520),
    (255, 1, 2, 512, 264), (257, 4, 5, 328, 392), (700, 1, 130, 136, 72), (1000, 2, 9, 192, 640),
    (2048, 1, 4, 320, 512), (3001, 2, 16, 256, 136),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_products(torch, shape, dtype):
    x_rows, share, E, K, N = shape
    x, dy, W, ids = problem(torch, 11, dtype, x_rows, share, E, K, N, pad=8)
    check_all(torch, x, dy, W, ids, share, dtype, "products", pad=16)


@pytest.mark.parametrize("kind", ["all in one", "none", "some outside", "last group only",
                                  "lengths around a tile"])
@pytest.mark.parametrize("rows", [48, 700])
def test_group_shapes(torch, kind, rows):
    E, K, N = 70, 264, 392
    rng = np.random.default_rng(3)
    if kind == "all in one":
        ids = np.full(rows, 66)
    elif kind == "none":
        ids = np.full(rows, -1)
    elif kind == "some outside":
        ids = rng.choice([-1, 0, 5, 69, 70, 1000], rows)
    elif kind == "last group only":
        ids = np.where(np.arange(rows) % 3 == 0, 69, -1)
    else:
        lens = [1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129] if rows > 64 else [1, 15, 16, 16]
        ids = rng.permutation(np.repeat(np.arange(len(lens)) * 3, lens))
        rows = len(ids)
    x, dy, W, ids = problem(torch, 12, "bf16", rows, 1, E, K, N, ids=ids)
    check_all(torch, x, dy, W, ids, 1, "bf16", kind)


@pytest.mark.parametrize("rows", [1, 3, 40, 300, 777])
def test_dense(torch, rows):
    """groups=None: one weight for all rows, in caller order."""
    import adapter_gemv_amd as sgmv
    K, N = 328, 264
    x, dy, W, _ = problem(torch, 13, "bf16", rows, 1, 1, K, N)
    W = W[0]
    y, dx, dW = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(W)
    sgmv.group_matmul(y, x, W)
    sgmv.group_matmul_dx(dx, dy, W)
    sgmv.group_matmul_dw(dW, x, dy)
    X, D, Wd, ids = f64(x), f64(dy), f64(W)[None], np.zeros(rows, int)
    close(f64(y), *G.group_matmul(X, Wd, ids), K, "bf16", "dense y")
    close(f64(dx), *G.group_matmul_dx(D, Wd, ids), N, "bf16", "dense dx")
    ref, mag = G.group_matmul_dw(X, D, ids, 1)
    close(f64(dW), ref[0], mag[0], rows, "bf16", "dense dW")


@pytest.mark.parametrize("rows", [24, 600])
def test_what_is_not_finite_stays_in_its_rows(torch, rows):
    """Infinities and NaN in rows of no group, in one group's rows or weights reach that
    group's outputs only."""
    import adapter_gemv_amd as sgmv
    E, K, N = 4, 264, 136
    ids = np.arange(rows) % 5 - 1                       # -1, 0, 1, 2, 3
    x, dy, W, ids_t = problem(torch, 14, "f16", rows, 1, E, K, N, ids=ids)
    clean_x, clean_dy, clean_W = x.clone(), dy.clone(), W.clone()
    for value in (float("nan"), float("inf")):
        x[ids_t == -1] = value
        dy[ids_t == -1] = value
        x[ids_t == 2] = value
        dy[ids_t == 2] = value
        W[2] = value
        groups = sgmv.group_rows(ids_t, E)
        y, dx, dW = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(W)
        sgmv.group_matmul(y, x, W, groups)
        sgmv.group_matmul_dx(dx, dy, W, groups)
        sgmv.group_matmul_dw(dW, x, dy, groups)
        keep = ids != 2
        X, D, Wd = f64(clean_x), f64(clean_dy), f64(clean_W)
        ref, mag = G.group_matmul(X, Wd, ids)
        close(f64(y)[keep], ref[keep], mag[keep], K, "f16", f"{value} y")
        ref, mag = G.group_matmul_dx(D, Wd, ids)
        close(f64(dx)[keep], ref[keep], mag[keep], N, "f16", f"{value} dx")
        ref, mag = G.group_matmul_dw(X, D, ids, E)
        close(f64(dW)[[0, 1, 3]], ref[[0, 1, 3]], mag[[0, 1, 3]], rows, "f16", f"{value} dW")
        assert not torch.isfinite(y[ids_t == 2]).any() and not torch.isfinite(dW[2]).any()


@pytest.mark.parametrize("rows,K,N", [(12, 24, 16), (90, 40, 72)])
def test_gradients_against_differences(torch, rows, K, N):
    """Whole numbers small enough that every product and sum is exact: the change of
    sum(c * y) when one element of x or W moves by one is that element's gradient, exactly."""
    import adapter_gemv_amd as sgmv
    E, share = 3, 2
    rng = np.random.default_rng(9)
    dev = lambda a: torch.tensor(a, dtype=torch.float16, device="cuda")  # noqa: E731
    x, W = rng.integers(-1, 2, (rows, K)), rng.integers(-1, 2, (E, N, K))
    c, ids = rng.integers(-1, 2, (rows * share, N)), rng.integers(-1, E, rows * share)
    groups = sgmv.group_rows(torch.tensor(ids, dtype=torch.int32, device="cuda"), E)

    def loss(xv, Wv):
        y = sgmv.group_matmul(dev(np.zeros((rows * share, N))), dev(xv), dev(Wv), groups)
        return float((y.double() * dev(c).double()).sum())

    dx = sgmv.group_matmul_dx(dev(np.zeros((rows * share, K))), dev(c), dev(W), groups)
    dx = dx.double().view(rows, share, K).sum(1).cpu().numpy()
    dW = f64(sgmv.group_matmul_dw(dev(W), dev(x), dev(c), groups))
    at = loss(x, W)
    for _ in range(25):
        i, k, g, o = rng.integers(rows), rng.integers(K), rng.integers(E), rng.integers(N)
        x2, W2 = x.copy(), W.copy()
        x2[i, k] += 1
        W2[g, o, k] += 1
        assert loss(x2, W) - at == dx[i, k]
        assert loss(x, W2) - at == dW[g, o, k]


@pytest.mark.parametrize("rows", [40, 1500])
def test_same_bits_every_time_and_under_graph_replay(torch, rows):
    import adapter_gemv_amd as sgmv
    E, share, K, N = 6, 2, 520, 264
    x, dy, W, ids = problem(torch, 15, "bf16", rows, share, E, K, N)
    n = rows * share

    def step():
        groups = sgmv.group_rows(ids, E)
        return (sgmv.group_matmul(torch.empty_like(dy), x, W, groups),
                sgmv.group_matmul_dx(x.new_empty(n, K), dy, W, groups),
                sgmv.group_matmul_dw(torch.empty_like(W), x, dy, groups))

    first = step()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(3):
            again = step()
            assert all(torch.equal(a, b) for a, b in zip(first, again))
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(3):
        ids.copy_((ids + r) % E)         # new groups for each replay
        want = step()
        for t in held:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), f"replay {r}"


def test_stream_argument(torch):
    import adapter_gemv_amd as sgmv
    x, dy, W, ids = problem(torch, 16, "bf16", 200, 1, 3, 264, 136)
    want = sgmv.group_matmul(torch.empty_like(dy), x, W, sgmv.group_rows(ids, 3))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = sgmv.group_matmul(torch.empty_like(dy), x, W, sgmv.group_rows(ids, 3, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows", [5, 300])
def test_rows_and_weights_past_32_bits(torch, rows):
    """Rows of x, dy, y and dx that end past 2^32 bytes from their base, and groups of W and
    dW 2^31 elements apart."""
    import adapter_gemv_amd as sgmv
    E, K, N = 2, 72, 136
    ld = ((1 << 31) + (1 << 26)) // (rows - 1) // 8 * 8
    t = torch.bfloat16
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    big = torch.zeros((rows - 1) * ld + 1024, dtype=t, device="cuda")
    view = lambda first, cols: big[first:].as_strided((rows, cols), (ld, 1))  # noqa: E731
    x, dy, y, dx = view(0, K), view(128, N), view(320, N), view(512, K)
    x.copy_(torch.randn(rows, K, generator=gen, device="cuda"))
    dy.copy_(torch.randn(rows, N, generator=gen, device="cuda") * N ** -0.5)
    # the outputs get a buffer of their own: strided views of one buffer overlap as ranges
    out = torch.zeros((rows - 1) * ld + 1024, dtype=t, device="cuda")
    y = out[320:].as_strided((rows, N), (ld, 1))
    dx = out[512:].as_strided((rows, K), (ld, 1))
    stride = (1 << 31) + 64
    pool = torch.zeros(stride + N * K, dtype=t, device="cuda")
    W = pool.as_strided((E, N, K), (stride, K, 1))
    W.copy_(torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5)
    ids = np.arange(rows) % 3 - 1
    groups = sgmv.group_rows(torch.tensor(ids, dtype=torch.int32, device="cuda"), E)
    say("past 32 bits")
    sgmv.group_matmul(y, x, W, groups)
    sgmv.group_matmul_dx(dx, dy, W, groups)
    X, D, Wd = f64(x), f64(dy), f64(W)
    close(f64(y), *G.group_matmul(X, Wd, ids), K, "bf16", "far y")
    close(f64(dx), *G.group_matmul_dx(D, Wd, ids), N, "bf16", "far dx")
    sgmv.group_matmul_dw(W, x, dy, groups)
    close(f64(W), *G.group_matmul_dw(X, D, ids, E), rows, "bf16", "far dW")


def test_no_rows(torch):
    import adapter_gemv_amd as sgmv
    W = torch.full((3, 16, 32), 5.0, dtype=torch.bfloat16, device="cuda")
    x, dy = W.new_empty(0, 32), W.new_empty(0, 16)
    groups = sgmv.group_rows(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert groups.starts.tolist() == [0, 0, 0, 0]
    assert sgmv.group_matmul(dy, x, W, groups).shape == (0, 16)
    sgmv.group_matmul_dw(W, x, dy, groups)
    assert not W.any()
