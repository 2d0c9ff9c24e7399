"""Microscaled 4-bit floating point on the GPU against the fp64 oracle: the format bit for
bit, the products within the rounding of their sums (as in the grouped products' tests)."""
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


def f64(t):
    return t.double().cpu().numpy()


def close(got, ref, mag, depth, dtype, what):
    u, sub = (2.0 ** -8, 2.0 ** -134) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)
    err = np.abs(got - ref)
    tol = u * np.abs(ref) + sub + (1 + u) * (depth + 32) * 2.0 ** -23 * mag
    say(f"{what}: max|err| {err.max():.3e}, worst err/tol {(err / tol).max():.3f}")
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} outside"


def same_values(torch, got, want64):
    """got holds exactly want64 rounded once to its type (NaN for NaN)."""
    want = torch.tensor(want64).to(torch.float32).to(got.dtype)   # 4-bit values are exact in float32
    g = got.cpu()
    both_nan = torch.isnan(g) & torch.isnan(want)
    assert torch.all(both_nan | (g == want)), f"{int((~(both_nan | (g == want))).sum())} differ"


# --------------------------------------------------------------------------------------
# the format
# --------------------------------------------------------------------------------------
def patterns(torch, dtype, seed):
    """Every 16-bit pattern once, in blocks of values of like size, of any size, and of one
    value among zeros."""
    rng = np.random.default_rng(seed)
    bits = np.arange(65536, dtype=np.uint16)
    like = bits[np.argsort(bits & 0x7fff, kind="stable")]          # neighbours in magnitude
    any_ = rng.permutation(bits)
    alone = np.zeros((2048, 32), np.uint16)
    alone[np.arange(2048), rng.integers(0, 32, 2048)] = bits[::32]
    both = np.concatenate([like, any_, alone.ravel()]).reshape(-1, 64)
    return torch.tensor(both.view(np.int16), device="cuda").view(_dt(torch, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_every_value(torch, dtype):
    import adapter_gemv_amd as sgmv
    x = patterns(torch, dtype, 1)
    q = sgmv.mx_quantize(x)
    codes, scales = G.mx_encode(f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    back = sgmv.mx_dequantize(torch.empty_like(x), q)
    same_values(torch, back, G.mx_decode(codes, scales))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_quantize_around_every_tie(torch, dtype):
    """Blocks whose largest value is 4, 6 or just below 8 times a power of two, with every
    value of the type between 0 and 8 times it."""
    import adapter_gemv_amd as sgmv
    for top in (4.0, 6.0, 7.96875):
        for power in (-12, 0, 9):
            one = torch.tensor(0.25, dtype=_dt(torch, dtype))
            lo, hi = 0, int(torch.tensor(7.96875, dtype=_dt(torch, dtype)).view(torch.int16))
            first = int(one.view(torch.int16)) - 256
            vals = torch.arange(max(lo, first), hi + 1, dtype=torch.int16).view(_dt(torch, dtype))
            vals = vals[vals <= top]
            pad = (-len(vals)) % 31
            vals = torch.cat([vals, torch.zeros(pad, dtype=vals.dtype)]).view(-1, 31)
            x = torch.cat([torch.full((len(vals), 1), top, dtype=vals.dtype), vals], 1)
            x = (x.double() * 2.0 ** power * torch.tensor([1.0, -1.0]).repeat(16)).to(vals.dtype).cuda()
            q = sgmv.mx_quantize(x)
            codes, scales = G.mx_encode(f64(x))
            assert np.array_equal(q.scales.cpu().numpy(), scales)
            assert np.array_equal(q.codes.cpu().numpy(), codes)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_dequantize_every_code_and_scale(torch, dtype):
    import adapter_gemv_amd as sgmv
    codes = np.tile(np.concatenate([np.arange(16) | (np.arange(16) << 4)]), (256, 1)).astype(np.uint8)
    scales = np.arange(256, dtype=np.uint8).reshape(256, 1)
    q = sgmv.MxTensor(torch.tensor(codes, device="cuda"), torch.tensor(scales, device="cuda"))
    y = torch.empty(256, 32, dtype=_dt(torch, dtype), device="cuda")
    same_values(torch, sgmv.mx_dequantize(y, q), G.mx_decode(codes, scales))


@pytest.mark.parametrize("rows,h,pad", [(1, 32, 0), (3, 96, 8), (17, 5120, 24), (1000, 64, 8), (5, 16416, 0)])
def test_quantize_rows_and_strides(torch, rows, h, pad):
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(rows)
    buf = torch.randn(rows, h + pad, generator=gen, device="cuda").to(torch.bfloat16)
    buf[:, h:] = float("nan")
    x = buf[:, :h]
    q = sgmv.mx_quantize(x)
    codes, scales = G.mx_encode(f64(x))
    assert np.array_equal(q.codes.cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
    out = torch.full_like(buf, 7.0)
    sgmv.mx_dequantize(out[:, :h], q)
    same_values(torch, out[:, :h], G.mx_decode(codes, scales))
    assert torch.all(out[:, h:] == 7.0)
    # one dimension and three
    assert torch.equal(sgmv.mx_quantize(x[0]).codes, q.codes[0])
    three = torch.stack([x, x * 2]).contiguous()
    assert torch.equal(sgmv.mx_quantize(three).scales[1], q.scales + (q.scales > 0).to(torch.uint8))
    assert sgmv.mx_quantize(x[:0]).codes.shape == (0, h // 2)


# --------------------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------------------
def weights(torch, gen, E, N, K, dtype):
    import adapter_gemv_amd as sgmv
    W = (torch.randn(E, N, K, generator=gen, device="cuda") * K ** -0.5).to(_dt(torch, dtype))
    return sgmv.mx_quantize(W)


def check(torch, x, q, ids, share, dtype, what, pad=8):
    """Both products through the public call, every element."""
    import adapter_gemv_amd as sgmv
    E, N, K = q.shape
    n = x.shape[0] * share
    ids_h = np.zeros(n, int) if ids is None else ids.cpu().numpy()
    groups = None if ids is None else sgmv.group_rows(ids, E)
    Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    say(f"{what}: n={n} share={share} E={E} K={K} N={N} {dtype}")
    for both in (False, True):
        buf = torch.full((n, N + pad), 7.0, dtype=x.dtype, device="cuda")
        xq = sgmv.mx_quantize(x) if both else x
        sgmv.mx_matmul(buf[:, :N], xq, q, groups)
        X = G.mx_decode(*G.mx_encode(f64(x))) if both else f64(x)
        ref, mag = G.group_matmul(X, Wd, ids_h, share)
        close(f64(buf[:, :N]), ref, mag, K, dtype, f"{what}, rows in {4 if both else 16} bits")
        assert torch.all(buf[:, N:] == 7.0), "padding written"


SHAPES = [
    # x rows, share, E (0: dense), K, N
    (1, 1, 0, 32, 8), (1, 1, 0, 4096, 264), (2, 2, 4, 64, 40), (5, 3, 9, 544, 136),
    (16, 1, 0, 256, 512), (17, 1, 3, 1056, 72), (33, 2, 8, 32, 1032), (64, 1, 0, 2080, 328),
    (65, 1, 0, 128, 64), (130, 2, 5, 288, 264), (300, 1, 0, 512, 520), (257, 4, 70, 96, 136),
    (1000, 1, 3, 320, 392), (2050, 1, 0, 256, 256),
]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_products(torch, shape, dtype):
    rows, share, E, K, N = shape
    gen = torch.Generator(device="cuda")
    gen.manual_seed(21)
    buf = torch.full((rows, K + 8), float("nan"), dtype=_dt(torch, dtype), device="cuda")
    x = buf[:, :K]
    x.copy_(torch.randn(rows, K, generator=gen, device="cuda"))
    q = weights(torch, gen, max(E, 1), N, K, dtype)
    ids = torch.randint(-1, E, (rows * share,), generator=gen, device="cuda", dtype=torch.int32) if E else None
    check(torch, x, q, ids, share, dtype, "mx")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("K", [256, 544, 96])
def test_enough_work_for_the_largest_tiles(torch, dtype, K):
    """Products that fill the card with 256 x 256 tiles, ragged groups, blocks that end inside a
    stage; every row against the oracle, 512 at a time."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(22)
    rows, E, N = 4300, 3, 4104
    x = torch.randn(rows, K, generator=gen, device="cuda").to(_dt(torch, dtype))
    q = weights(torch, gen, E, N, K, dtype)
    q.scales[0, 7] = 90                                  # float16 does not hold these weights
    ids = torch.randint(-1, E, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    groups, ids_h = sgmv.group_rows(ids, E), ids.cpu().numpy()
    Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    for both in (False, True):
        y = sgmv.mx_matmul(torch.empty(rows, N, dtype=x.dtype, device="cuda"),
                           sgmv.mx_quantize(x) if both else x, q, groups)
        X = G.mx_decode(*G.mx_encode(f64(x))) if both else f64(x)
        for lo in range(0, rows, 512):
            part = slice(lo, min(rows, lo + 512))
            ref, mag = G.group_matmul(X[part], Wd, ids_h[part])
            close(f64(y[part]), ref, mag, K, dtype, f"both {both} rows {lo}..")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("E,K", [(0, 96), (0, 512), (7, 160), (40, 288)])
def test_enough_work_for_half_of_the_largest_tiles(torch, dtype, E, K):
    """Products of about one round of 128 x 256 tiles, from one group of whole tiles to 40 ragged
    ones with rows of none; every row against the oracle, 512 at a time."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(23)
    rows, N = 1100, 7000 if E == 0 else 5000 if E == 7 else 1544
    x = torch.randn(rows, K, generator=gen, device="cuda").to(_dt(torch, dtype))
    q = weights(torch, gen, max(E, 1), N, K, dtype)
    if E == 0:
        q = sgmv.MxTensor(q.codes[0], q.scales[0])
    ids = torch.randint(-1, E, (rows,), generator=gen, device="cuda", dtype=torch.int32) if E else None
    groups = sgmv.group_rows(ids, E) if E else None
    Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    y = sgmv.mx_matmul(torch.full((rows, N), float("nan"), dtype=x.dtype, device="cuda"), x, q, groups)
    for lo in range(0, rows, 512):
        part = slice(lo, min(rows, lo + 512))
        ref, mag = G.group_matmul(f64(x[part]), Wd if E else Wd[None],
                                  ids[part].cpu().numpy() if E else np.zeros(part.stop - lo, np.int32))
        close(f64(y[part]), ref, mag, K, dtype, f"rows {lo}..")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [20, 150])
@pytest.mark.parametrize("K", [8192, 8224, 8416])
def test_few_rows_of_long_weights(torch, dtype, rows, K):
    """Decode batches over enough long rows that a wavefront makes several rounds, with scales of
    a row that start at any byte; x in 16 and in 4 bits."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(24)
    E, N = 8, 1064
    x = torch.randn(rows, K, generator=gen, device="cuda").to(_dt(torch, dtype))
    q = weights(torch, gen, E, N, K, dtype)
    ids = torch.randint(-1, E, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    groups = sgmv.group_rows(ids, E)
    Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    for both in (False, True):
        y = sgmv.mx_matmul(torch.full((rows, N), float("nan"), dtype=x.dtype, device="cuda"),
                           sgmv.mx_quantize(x) if both else x, q, groups)
        ref, mag = G.group_matmul(G.mx_decode(*G.mx_encode(f64(x))) if both else f64(x), Wd, ids.cpu().numpy())
        close(f64(y), ref, mag, K, dtype, f"both {both}")


@pytest.mark.parametrize("rows", [3, 40, 200, 3000])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("low", [1, 60, 118, 140])
def test_scales_of_any_size(torch, rows, dtype, low):
    """Scales from `low` to `low` + 20 (powers of two that float16 does not hold), with x of
    the size that makes the sums of ordinary size where its type can: no weight is lost or
    overflows on its way to the product."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(low)
    K, N = 160, 136
    codes = torch.randint(0, 256, (1, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    scales = torch.randint(low, low + 21, (1, N, K // 32), generator=gen, device="cuda", dtype=torch.uint8)
    q = sgmv.MxTensor(codes, scales)
    limit = 14 if dtype == "f16" else 120
    power = max(-limit, min(limit, 127 - low - 20))
    x = (torch.randn(rows, K, generator=gen, device="cuda") * 2.0 ** power).to(_dt(torch, dtype))
    y = sgmv.mx_matmul(torch.empty(rows, N, dtype=x.dtype, device="cuda"), x, q)
    with np.errstate(invalid="ignore"):
        ref, mag = G.group_matmul(f64(x), G.mx_decode(codes.cpu().numpy(), scales.cpu().numpy()),
                                  np.zeros(rows, int))
    got = f64(y)
    # x of size 2^14 in float16 holds a few infinities: their rows are infinite or NaN (an
    # infinity times a zero code) on both sides
    odd = ~np.isfinite(ref)
    assert np.array_equal(got[odd], ref[odd], equal_nan=True)
    most = 65504.0 if dtype == "f16" else 3.3e38
    assert np.isinf(got[~odd & (np.abs(np.where(odd, 0, ref)) > 1.01 * most)]).all()
    ok = ~odd & (np.abs(np.where(odd, 0, ref)) < 0.99 * most)
    if ok.any():
        close(got[ok], ref[ok], mag[ok], K, dtype, f"scales from {low}")


@pytest.mark.parametrize("rows", [4, 300])
def test_nan_scale_and_infinite_rows_stay_where_they_are(torch, rows):
    """A block scaled by NaN makes its own output column NaN and no other; an infinity in x
    reaches its own row only, one in a row of no group none."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(31)
    E, K, N = 3, 288, 72
    q = weights(torch, gen, E, N, K, "bf16")
    x = torch.randn(rows, K, generator=gen, device="cuda").to(torch.bfloat16)
    ids_h = np.arange(rows) % 4 - 1
    ids = torch.tensor(ids_h, dtype=torch.int32, device="cuda")
    groups = sgmv.group_rows(ids, E)
    Wd = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())
    q.scales[1, 5, 8] = 255
    q.scales[1, 71, 0] = 255
    x2 = x.clone()
    x2[0, 3] = float("inf")                              # a row of no group
    x2[3, 7] = float("inf")                              # a row of group 2
    for both in (False, True):
        y = sgmv.mx_matmul(torch.empty(rows, N, dtype=x.dtype, device="cuda"),
                           sgmv.mx_quantize(x2) if both else x2, q, groups)
        got = f64(y)
        X = G.mx_decode(*G.mx_encode(f64(x))) if both else f64(x)
        ref, mag = G.group_matmul(X, Wd, ids_h)
        bad = np.zeros(ref.shape, bool)
        bad[np.ix_(ids_h == 1, [5, 71])] = True
        assert np.isnan(got[bad]).all()
        assert not np.isfinite(got[3]).any()
        bad[3] = True
        close(np.where(bad, 0, got), np.where(bad, 0, ref), np.where(bad, 0, mag), K, "bf16", "others")


@pytest.mark.parametrize("rows", [8, 600])
def test_same_bits_and_graph_replay(torch, rows):
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(41)
    E, K, N = 4, 544, 264
    q = weights(torch, gen, E, N, K, "f16")
    x = torch.randn(rows, K, generator=gen, device="cuda").half()
    ids = torch.randint(0, E, (rows,), generator=gen, device="cuda", dtype=torch.int32)

    def step():
        groups = sgmv.group_rows(ids, E)
        y = torch.empty(rows, N, dtype=x.dtype, device="cuda")
        return sgmv.mx_matmul(y, x, q, groups), sgmv.mx_matmul(torch.empty_like(y), sgmv.mx_quantize(x), q, groups)

    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, step()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for r in range(3):
        x.mul_(-1.5)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), f"replay {r}"
