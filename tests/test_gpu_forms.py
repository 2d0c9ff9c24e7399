"""Each form of the grouped and 4-bit kernels, at sizes that take it (form_sizes.py), against the
fp64 oracle with the tolerances of the grouped products' tests: rows of no group, what is not
finite, far strides, the same bits every time, graph replay."""
import numpy as np
import pytest

import form_sizes as F
from oracle import grouped_oracle as G
from test_gpu_grouped import close, f64, padded, say
from test_gpu_mx_scales import close as close_or_over      # infinite where the type ends

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def _type(torch, dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


def make(torch, size, dtype, seed=51, kind="mixed"):
    """(x, W, ids on the device or None, ids for the oracle) of a size; ids outside [0, groups) too."""
    rows, share, E, K, N = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = _type(torch, dtype)
    n = rows * share
    x, _ = padded(torch, rows, K, t, 8, gen)
    W = (torch.randn(max(E, 1), N, K, generator=gen, device="cuda") * K ** -0.5).to(t)
    if E == 0:
        return x, W, None, np.zeros(n, int)
    rng = np.random.default_rng(seed)
    if kind == "none":
        ids = rng.choice([-1, E, 2 ** 31 - 1, -2 ** 31], n)
    elif kind == "last":
        ids = np.where(np.arange(n) % 4 == 1, -1, E - 1)
    else:
        ids = rng.choice(np.r_[np.arange(E), np.arange(E), -1, E + 5], n)
    return x, W, torch.tensor(ids, dtype=torch.int32, device="cuda"), ids


def out(torch, n, N, dtype, pad=8):
    buf = torch.full((n, N + pad), 7.0, dtype=_type(torch, dtype), device="cuda")
    return buf[:, :N], buf


def product(torch, size, x, W, ids, **kw):
    """The public call on either kind of weight."""
    import adapter_gemv_amd as sgmv
    groups = None if ids is None else sgmv.group_rows(ids, size[2])
    y = torch.full((size[0] * size[1], size[4]), float("nan"), dtype=kw.pop("dtype", getattr(x, "dtype", None)),
                   device="cuda")
    call = sgmv.mx_matmul if isinstance(W, sgmv.MxTensor) else sgmv.group_matmul
    return call(y, x, W, groups, **kw)


# --------------------------------------------------------------------------------------
# 16-bit weights, streamed
# --------------------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", F.STREAMED, ids=lambda s: "x".join(map(str, s)))
def test_streamed(torch, size, dtype):
    import adapter_gemv_amd as sgmv
    rows, share, E, K, N = size
    for kind in ("mixed", "last", "none") if E else ("mixed",):
        x, W, ids, ids_h = make(torch, size, dtype, kind=kind)
        y, buf = out(torch, rows * share, N, dtype)
        say(f"streamed {size} {dtype} {kind}")
        sgmv.group_matmul(y, x, W, None if ids is None else sgmv.group_rows(ids, E))
        close(f64(y), *G.group_matmul(f64(x), f64(W), ids_h, share), K, dtype, f"{size} {kind}")
        assert torch.all(buf[:, N:] == 7.0), "padding written"
        assert not y[torch.tensor((ids_h < 0) | (ids_h >= max(E, 1)), device="cuda")].any()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", F.STREAMED_MIXED, ids=lambda s: "x".join(map(str, s)))
def test_streamed_what_is_not_finite_stays_in_its_rows(torch, size, dtype):
    rows, share, E, K, N = size
    x, W, _, _ = make(torch, size, dtype)
    x = x.clone()
    ids_h = np.arange(rows) % 5 - 1
    ids = torch.tensor(ids_h, dtype=torch.int32, device="cuda")
    ref, mag = G.group_matmul(f64(x), f64(W), ids_h)
    one = int(np.flatnonzero(ids_h == 0)[0])
    for value in (float("nan"), float("inf"), float("-inf")):
        x[ids == -1] = value
        x[ids == 2] = value
        W[2] = value
        x[one, K - 1] = value                              # a row among finite ones of its group
        W[1, N - 1, 0] = value                             # a column
        y = f64(product(torch, size, x, W, ids))
        bad = np.zeros(ref.shape, bool)
        bad[ids_h == 2] = True
        bad[one] = True
        bad[np.ix_(ids_h == 1, [N - 1])] = True
        assert not np.isfinite(y[bad]).any()
        close(np.where(bad, 0, y), np.where(bad, 0, ref), np.where(bad, 0, mag), K, dtype, f"{value}")


def test_streamed_past_32_bits(torch):
    """Rows of x and y that end past 2^32 bytes from their base, groups of W 2^31 elements apart."""
    import adapter_gemv_amd as sgmv
    rows, _, E, K, N = F.STREAMED_FAR
    ld = ((1 << 31) + (1 << 26)) // (rows - 1) // 8 * 8
    t = torch.bfloat16
    x = torch.zeros((rows - 1) * ld + 2048, dtype=t, device="cuda")[:].as_strided((rows, K), (ld, 1))
    y = torch.zeros((rows - 1) * ld + 2048, dtype=t, device="cuda")[:].as_strided((rows, N), (ld, 1))
    stride = (1 << 31) + 64
    W = torch.zeros(stride + N * K, dtype=t, device="cuda").as_strided((E, N, K), (stride, K, 1))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(6)
    x.copy_(torch.randn(rows, K, generator=gen, device="cuda"))
    W.copy_(torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5)
    ids = np.array([1, -1, 0, 1, 1])
    say("streamed past 32 bits")
    sgmv.group_matmul(y, x, W, sgmv.group_rows(torch.tensor(ids, dtype=torch.int32, device="cuda"), E))
    close(f64(y), *G.group_matmul(f64(x), f64(W), ids), K, "bf16", "far")


def replayed(torch, step, change):
    """`step` makes the same bits each time, on another stream, and from a captured graph, whatever
    `change` does to its inputs between the replays."""
    first = step().clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(5):
            assert torch.equal(first, step())
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(4):
        change(r)
        want = step()
        held.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want, held), f"replay {r}"


@pytest.mark.parametrize("size", F.STREAMED_REPEATED, ids=lambda s: "x".join(map(str, s)))
def test_streamed_same_bits_and_graph_replay(torch, size):
    x, W, ids, _ = make(torch, size, "bf16")
    ids.clamp_(0, size[2] - 1)

    def change(r):
        x.mul_(-1.25)
        ids.copy_((ids + r) % size[2])

    replayed(torch, lambda: product(torch, size, x, W, ids), change)


# --------------------------------------------------------------------------------------
# 4-bit weights, in every form
# --------------------------------------------------------------------------------------
MX = [*F.MX_DEEP, *F.MX_WIDE, *F.BOTH_DEEP, *F.BOTH_WIDE, *(s for sizes in F.MX_TILES.values() for s in sizes)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", MX, ids=lambda s: "x".join(map(str, s)))
def test_mx(torch, size, dtype):
    """Scales about the ends of those that float16 holds (2^-23 .. 2^13), in the first, a middle and the
    last block of some rows or throughout; x in 16 and in 4 bits; rows of no group."""
    import adapter_gemv_amd as sgmv
    rows, share, E, K, N = size
    x, W, ids, ids_h = make(torch, size, dtype, seed=52)
    q = sgmv.mx_quantize(W)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(53)
    blocks = K // 32
    for what in ("ordinary", "some", "all"):
        if what == "some":
            for i, b in enumerate((0, blocks // 2, blocks - 1)):
                q.scales[:, i::5, b] = 103 if i == 1 else 141
        elif what == "all":
            q.scales.copy_(torch.randint(96, 146, q.scales.shape, generator=gen, device="cuda"))
        Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
        xs = x * 2.0 ** -12 if what == "all" else x
        for both in (False, True):
            say(f"mx {size} {dtype} {what} both {both}")
            y = product(torch, size, sgmv.mx_quantize(xs) if both else xs, q if E else sgmv.MxTensor(
                q.codes[0], q.scales[0]), ids, dtype=x.dtype)
            X = G.mx_decode(*G.mx_encode(f64(xs))) if both else f64(xs)
            for lo in range(0, rows * share, 512 * share):
                part = slice(lo, lo + 512 * share)
                ref, mag = G.group_matmul(X[lo // share:lo // share + 512], Wd, ids_h[part], share)
                close_or_over(f64(y[part]), ref, mag, K, dtype, f"{what} both {both} rows {lo}..")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("size", [s for s in MX if s[2]], ids=lambda s: "x".join(map(str, s)))
def test_mx_what_is_not_finite_stays_where_it_is(torch, size, dtype):
    """A block scaled by NaN makes its own output column NaN, an infinity in x its own row not
    finite; rows of no group and other groups see neither."""
    import adapter_gemv_amd as sgmv
    rows, share, E, K, N = size
    x, W, _, _ = make(torch, size, dtype, seed=54)
    x = x.clone()
    ids_h = np.arange(rows * share) % (E + 1) - 1
    ids = torch.tensor(ids_h, dtype=torch.int32, device="cuda")
    q = sgmv.mx_quantize(W)
    Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    clean = x.clone()
    q.scales[1, 5, K // 32 - 1] = 255
    q.scales[1, N - 1, 0] = 255
    x[rows - 1, 7] = float("inf")                          # rows - 1 of x: the last `share` rows
    for both in (False, True):
        y = f64(product(torch, size, sgmv.mx_quantize(x) if both else x, q, ids, dtype=x.dtype))
        X = G.mx_decode(*G.mx_encode(f64(clean))) if both else f64(clean)
        nan = np.zeros(y.shape, bool)
        nan[np.ix_(ids_h == 1, [5, N - 1])] = True
        assert np.isnan(y[nan]).all()
        last = np.zeros(y.shape, bool)
        last[-share:] = ids_h[-share:, None] >= 0
        assert not np.isfinite(y[last]).any()
        bad = nan | last
        for lo in range(0, rows * share, 512 * share):
            part = slice(lo, lo + 512 * share)
            ref, mag = G.group_matmul(X[lo // share:lo // share + 512], Wd, ids_h[part], share)
            keep = ~bad[part]
            close(np.where(keep, y[part], 0), np.where(keep, ref, 0), np.where(keep, mag, 0), K, dtype,
                  f"both {both} rows {lo}..")


@pytest.mark.parametrize("both", [False, True], ids=["x16", "x4"])
@pytest.mark.parametrize("size", [F.MX_DEEP[2], F.MX_WIDE[1], F.MX_TILES[F.TILE_256][1], F.BOTH_DEEP[2],
                                  F.BOTH_WIDE[0]],
                         ids=lambda s: "x".join(map(str, s)))
def test_mx_same_bits_and_graph_replay(torch, size, both):
    import adapter_gemv_amd as sgmv
    x, W, ids, _ = make(torch, size, "f16", seed=55)
    ids.clamp_(0, size[2] - 1)
    q = sgmv.mx_quantize(W)
    q.scales[0, 3, 1] = 100                                # float16 does not hold these weights

    def change(r):
        x.mul_(-1.25)
        ids.copy_((ids + r) % size[2])

    replayed(torch, lambda: product(torch, size, sgmv.mx_quantize(x) if both else x, q, ids, dtype=x.dtype), change)


# --------------------------------------------------------------------------------------
# the stream argument
# --------------------------------------------------------------------------------------
CALLS = ["group_rows", "group_matmul", "group_matmul_dx", "group_matmul_dw", "mx_quantize", "mx_dequantize",
         "mx_matmul", "mx_matmul both"]


@pytest.mark.parametrize("name", CALLS)
def test_work_goes_to_the_stream_that_is_given(torch, name):
    """A call on a stream that is being captured becomes part of the graph, though the current stream
    is another one: replays write its output."""
    import adapter_gemv_amd as sgmv
    rows, E, K, N = 40, 3, 288, 136
    gen = torch.Generator(device="cuda")
    gen.manual_seed(61)
    x = torch.randn(rows, K, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(rows, N, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5).bfloat16()
    ids = torch.randint(-1, E, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    groups, q, xq = sgmv.group_rows(ids, E), sgmv.mx_quantize(W), sgmv.mx_quantize(x)
    new = lambda *shape: torch.full(shape, 9.0, dtype=x.dtype, device="cuda")  # noqa: E731
    outs = {"group_matmul": new(rows, N), "group_matmul_dx": new(rows, K), "group_matmul_dw": new(E, N, K),
            "mx_dequantize": new(E, N, K), "mx_matmul": new(rows, N), "mx_matmul both": new(rows, N)}

    def call(y, **kw):
        if name == "group_rows":
            return sgmv.group_rows(ids, E, **kw).table
        if name == "group_matmul":
            return sgmv.group_matmul(y, x, W, groups, **kw)
        if name == "group_matmul_dx":
            return sgmv.group_matmul_dx(y, dy, W, groups, **kw)
        if name == "group_matmul_dw":
            return sgmv.group_matmul_dw(y, x, dy, groups, **kw)
        if name == "mx_quantize":
            made = sgmv.mx_quantize(x, **kw)
            return made.codes
        if name == "mx_dequantize":
            return sgmv.mx_dequantize(y, q, **kw)
        return sgmv.mx_matmul(y, xq if name.endswith("both") else x, q, groups, **kw)

    y = outs.get(name)
    want = call(None if y is None else torch.empty_like(y)).cpu()
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        graph.capture_begin(capture_error_mode="relaxed")
    got = call(y, stream=stream)                           # the current stream is another one
    with torch.cuda.stream(stream):
        graph.capture_end()
    for _ in range(3):
        got.fill_(5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got.cpu(), want)
