"""8-bit floating point with a scale for each block of 128, and products in it, against the fp64
oracle.  Codes, scales and dequantised values are compared for equality.

Tolerance of a product: its own rounding to 16 bits (half a step, and half the smallest subnormal), and
the float32 sum's: every product of a block is exact in float32, and is summed, scaled and summed
again with at most one rounding or truncation (2^-23 of the magnitudes) a step, (depth + 32) steps.

The matrix instruction adds eight products at a time, and of these it cuts off, towards zero, what lies
below 2^-13 of the power of two that the largest one's exponents make (measured: beside 2^16, 8 stays
and 7 goes, and 26 becomes 24; the sums of eight are joined in float32).  That power is at most the largest
of the eight magnitudes, so at most seven products lose less than 2^-13 of it each: over all eights no more
than 7 * 2^-13 of the magnitudes' sum (CUT).  Where every value's exponent is one of three next to each other
nothing is lost: products are multiples of 2^(2 e - 6), for e the least exponent, and what is kept goes down
to 2^(2 (e + 2) - 13) = 2^(2 e - 9).  Those ("narrow") values are held to the float32 sum's tolerance alone."""
import numpy as np
import pytest

import block_sizes
from oracle import block_oracle as B
from oracle import grouped_oracle as G

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def f64(t):
    return t.double().cpu().numpy()


def codes_of(t, torch):
    return t.view(torch.uint8).cpu().numpy()


def kind(torch, dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float16


CUT = 7 * 2.0 ** -13


def close(got, ref, mag, depth, dtype, what, narrow=False):
    u, sub = (2.0 ** -8, 2.0 ** -134) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)
    tol = u * np.abs(ref) + sub + (1 + u) * ((depth + 32) * 2.0 ** -23 + (0 if narrow else CUT)) * mag
    err = np.abs(got - ref)
    print(f"{what}: worst err/tol {(err / tol).max() if err.size else 0:.3f}", flush=True)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} outside"


def strided(torch, v, pad):
    """v as a view of a buffer with `pad` more columns that hold NaN."""
    store = torch.full((*v.shape[:-1], v.shape[-1] + pad), float("nan"), dtype=v.dtype, device="cuda")
    store[..., :v.shape[-1]] = v
    return store[..., :v.shape[-1]]


# --------------------------------------------------------------------------------------
# quantisation
# --------------------------------------------------------------------------------------
def values(torch, dtype, shape, seed):
    """Values of every size, rows and columns apart, with zeros, blocks of zeros and the type's ends."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    v = torch.randn(*shape, generator=gen, device="cuda")
    span = 120.0 if dtype == "bf16" else 12.0
    v = v * torch.exp2((torch.rand(shape[0], 1, generator=gen, device="cuda") * 2 - 1) * span)
    v = v * torch.exp2(-40 * torch.rand(1, shape[1], generator=gen, device="cuda") ** 8)
    v = v.to(kind(torch, dtype))
    v[torch.rand(*shape, generator=gen, device="cuda") < 0.05] = 0.0
    v[:, :128][::5] = 0.0
    v[1::7] *= -0.0
    return v


@pytest.mark.parametrize("shape", [(1, 16), (3, 128), (5, 144), (300, 272), (7, 2048), (2, 5136), (129, 1040)], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_and_back(torch, shape, dtype):
    import adapter_gemv_amd as sgmv
    v = values(torch, dtype, shape, sum(shape))
    v[0, 0] = torch.finfo(v.dtype).max
    codes, scales = B.encode(f64(v), 1)
    for x in (v, strided(torch, v, 24)):
        q = sgmv.fp8_quantize(x)
        assert np.array_equal(f64(q.scales), scales) and np.array_equal(codes_of(q.codes, torch), codes)
        back = sgmv.fp8_dequantize(torch.empty_like(x), q)
        want = torch.tensor(B.decode(codes, scales, 1)).to(v.dtype)
        assert torch.equal(back.cpu(), want)


@pytest.mark.parametrize("shape", [(1, 16, 16), (1, 128, 128), (3, 144, 272), (2, 1040, 528), (1, 2048, 16), (5, 16, 400),
                                   (3, 136, 272), (2, 8, 16)],
                         ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_and_back(torch, shape, dtype):
    import adapter_gemv_amd as sgmv
    E, N, K = shape
    v = torch.stack([values(torch, dtype, (N, K), e + N) for e in range(E)])
    parts = [B.encode(f64(w), 128) for w in v]
    room = torch.full((E, N * K + 40), float("nan"), dtype=v.dtype, device="cuda")
    apart = room.as_strided((E, N, K), (N * K + 40, K, 1)) if E > 1 else v.clone()
    apart.copy_(v)
    for W in (v, apart, *([v[0]] if E == 1 else [])):
        q = sgmv.fp8_quantize_weight(W)
        assert q.shape == tuple(W.shape)
        got, s = codes_of(q.codes, torch).reshape(E, N, K), f64(q.scales).reshape(E, -(-N // 128), -(-K // 128))
        for e, (codes, scales) in enumerate(parts):
            assert np.array_equal(got[e], codes) and np.array_equal(s[e], scales)
        back = sgmv.fp8_dequantize(torch.empty_like(v).view(W.shape) if W is not apart else apart.clone(), q)
        want = np.stack([B.decode(c, sc, 128) for c, sc in parts]).reshape(tuple(W.shape))
        assert torch.equal(back.cpu(), torch.tensor(want).to(v.dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_16_bit_value(torch, dtype):
    """Each finite value of the type beside each of a few largest elements: every rounding, subnormal codes and
    scales at the end of the range."""
    import adapter_gemv_amd as sgmv
    t = kind(torch, dtype)
    every = torch.arange(65536, device="cuda").to(torch.int32).to(torch.int16).view(t)
    every = every[torch.isfinite(every)]
    every = every[every.abs().sort().indices]
    for top in (1.0, 1.75, 1.76, 448.0, 449.0, 2.0 ** -14, float(torch.finfo(t).max), float(torch.finfo(t).tiny), 0.0):
        fits = every[every.abs() <= top]
        fits = torch.cat([fits, fits.new_zeros(-fits.numel() % 127)]).view(-1, 127)
        x = torch.cat([torch.full_like(fits[:, :1], top), fits], 1)
        q = sgmv.fp8_quantize(x)
        codes, scales = B.encode(f64(x), 1)
        assert np.array_equal(f64(q.scales), scales), top
        assert np.array_equal(codes_of(q.codes, torch), codes), top


def test_every_code_times_scales(torch):
    """Dequantised values are rounded once, also where float32 does not hold the product, in the type's subnormals
    and past its end."""
    import adapter_gemv_amd as sgmv
    from fractions import Fraction
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    scales = torch.cat([torch.rand(40, generator=gen, device="cuda") + 0.5,
                        torch.exp2(torch.randint(-149, 128, (80,), generator=gen, device="cuda").double()).float(),
                        torch.rand(40, generator=gen, device="cuda") * 2.0 ** -20,
                        torch.tensor([0.0, float("inf"), float("nan"), -1.5, 1 + 2.0 ** -8, 1 + 2.0 ** -11 + 2.0 ** -23,
                                      (1 + 2.0 ** -9) * (1 - 2.0 ** -24)], device="cuda")])
    all_codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 2, 128).expand(scales.numel(), 2, 128)
    q = sgmv.Fp8Rows(all_codes.reshape(-1, 256).contiguous().view(torch.float8_e4m3fn), scales[:, None].repeat(1, 2))
    exact = B.decode(codes_of(q.codes, torch), f64(q.scales), 1)
    for dtype in ("bf16", "f16"):
        got = sgmv.fp8_dequantize(torch.empty(q.shape, dtype=kind(torch, dtype), device="cuda"), q).cpu()
        # numpy and torch round float64 to 16 bits by way of float32: round here, by whole numbers of steps
        bits, low, most = (8, -133, float(torch.finfo(torch.bfloat16).max)) if dtype == "bf16" else (11, -24, 65504.0)
        want = np.array(exact)
        ok = np.isfinite(exact) & (exact != 0)
        m, e = np.frexp(exact[ok])
        step = np.maximum(e - bits, low)
        r = np.array([float(Fraction(v) / Fraction(2) ** int(s)) for v, s in zip(exact[ok], step)])
        r = np.ldexp(np.round(r), step)
        want[ok] = np.where(np.abs(r) > most, np.copysign(np.inf, r), r)
        g = f64(got)
        assert np.array_equal(np.isnan(g), np.isnan(want)) and np.array_equal(g[~np.isnan(g)], want[~np.isnan(want)])


def test_blocks_that_are_not_finite(torch):
    import adapter_gemv_amd as sgmv
    for t in (torch.bfloat16, torch.float16):
        x = torch.ones(6, 400, dtype=t, device="cuda")
        x[0, 5], x[1, 399], x[2, 130] = float("inf"), float("nan"), -float("inf")
        q = sgmv.fp8_quantize(x)
        bad = torch.isnan(q.scales).nonzero().tolist()
        assert bad == [[0, 0], [1, 3], [2, 1]]
        assert not q.codes.view(torch.uint8)[0, :128].any() and not q.codes.view(torch.uint8)[1, 384:].any()
        back = sgmv.fp8_dequantize(torch.empty_like(x), q)
        assert torch.isnan(back).sum() == 128 + 16 + 128 and bool((back[~torch.isnan(back)] == 1).all())
        W = torch.ones(3, 144, 144, dtype=t, device="cuda")
        W[1, 140, 3] = float("nan")
        qw = sgmv.fp8_quantize_weight(W)
        assert torch.isnan(qw.scales).nonzero().tolist() == [[1, 1, 0]]


# --------------------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------------------
def weight(torch, gen, E, N, K):
    """Codes of every kind but NaN, and scales that are no powers of two."""
    import adapter_gemv_amd as sgmv
    codes = torch.randint(0, 254, (E, N, K), generator=gen, device="cuda", dtype=torch.int32)
    codes = torch.where(codes >= 127, codes + 1, codes).to(torch.uint8)
    scales = torch.exp(torch.randn(E, -(-N // 128), -(-K // 128), generator=gen, device="cuda")) * K ** -0.5 / 200
    return sgmv.Fp8Weight(codes.view(torch.float8_e4m3fn), scales)


def rows(torch, gen, n, h, dtype, pad):
    v = torch.randn(n, h, generator=gen, device="cuda") * torch.exp(torch.randn(n, 1, generator=gen, device="cuda"))
    return strided(torch, v.to(kind(torch, dtype)), pad)


def narrow_values(torch, gen, *shape):
    """Eight mantissas, three exponents, both signs: exact in 8 bits wherever they stand."""
    m = torch.randint(8, 16, shape, generator=gen, device="cuda").float() / 8
    e = torch.randint(0, 3, shape, generator=gen, device="cuda").float()
    s = torch.randint(0, 2, shape, generator=gen, device="cuda").float() * 2 - 1
    return m * torch.exp2(e) * s


def narrow_weight(torch, gen, E, N, K):
    import adapter_gemv_amd as sgmv
    codes = narrow_values(torch, gen, E, N, K).to(torch.float8_e4m3fn)
    return sgmv.Fp8Weight(codes, torch.exp(torch.randn(E, -(-N // 128), -(-K // 128), generator=gen, device="cuda")) * K ** -0.5)


def narrow_rows(torch, gen, n, h, dtype, pad):
    v = narrow_values(torch, gen, n, h) * torch.exp2(torch.randint(-3, 4, (n, 1), generator=gen, device="cuda").float())
    return strided(torch, v.to(kind(torch, dtype)), pad)


def check(torch, T, share, E, K, N, dtype, seed=0, ids=None, pad=0, grouped=True, dx=True, forward=True, narrow=False):
    """Both products through the public calls, 16-bit rows and rows taken to 8 bits before."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n = T * share
    weight, rows = (narrow_weight, narrow_rows) if narrow else (globals()["weight"], globals()["rows"])
    W = weight(torch, gen, E, N, K)
    Wd = np.stack([B.decode(c, s, 128) for c, s in zip(codes_of(W.codes, torch), f64(W.scales))])
    groups = None
    if grouped:
        ids = torch.randint(-1, E + 1, (n,), generator=gen, device="cuda", dtype=torch.int32) if ids is None else \
            torch.tensor(ids, dtype=torch.int32, device="cuda")
        groups = sgmv.group_rows(ids, E)
    at = ids.cpu().numpy() if grouped else np.zeros(n, int)
    what = f"{T}x{share} of {E}, {K} x {N} {dtype}"
    if forward:
        x = rows(torch, gen, T, K, dtype, pad)
        ref, mag = G.group_matmul(B.decode(*B.encode(f64(x), 1), 1), Wd, at, share)
        out = strided(torch, torch.empty(n, N, dtype=x.dtype, device="cuda"), pad)
        y = sgmv.fp8_matmul(out, x, W, groups)
        assert y is out
        close(f64(y), ref, mag, K, dtype, what, narrow)
        y8 = sgmv.fp8_matmul(torch.full_like(y.contiguous(), float("nan")), sgmv.fp8_quantize(x), W, groups)
        close(f64(y8), ref, mag, K, dtype, what + " from 8 bits", narrow)
        assert torch.equal(y, y8)
    if dx:
        dy = rows(torch, gen, n, N, dtype, pad)
        ref, mag = G.group_matmul_dx(B.decode(*B.encode(f64(dy), 1), 1), Wd, at)
        out = strided(torch, torch.empty(n, K, dtype=dy.dtype, device="cuda"), pad)
        d = sgmv.fp8_matmul_dx(out, dy, W, groups)
        assert d is out
        close(f64(d), ref, mag, N, dtype, what + " dx", narrow)
        if N % 16 == 0:
            d8 = sgmv.fp8_matmul_dx(torch.full_like(d.contiguous(), float("nan")), sgmv.fp8_quantize(dy), W, groups)
            assert torch.equal(d, d8)


DENSE = [(1, 16, 16), (1, 128, 128), (1, 4096, 1024), (3, 144, 272), (16, 1040, 528), (17, 272, 144), (33, 2064, 400),
         (64, 512, 640), (65, 400, 2064), (129, 1040, 528), (300, 656, 784), (513, 272, 1168), (1000, 144, 144)]


@pytest.mark.parametrize("size", DENSE, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("narrow", [True, False])
def test_dense(torch, size, dtype, narrow):
    T, K, N = size
    check(torch, T, 1, 1, K, N, dtype, seed=T, grouped=False, narrow=narrow)


ODD = [(1, 1, 1, 16, 8), (5, 2, 3, 144, 136), (40, 1, 1, 272, 520), (300, 2, 2, 400, 264), (2100, 1, 3, 1040, 1032),
       (2050, 1, 1, 640, 4104), (1111, 1, 1, 4112, 648)]


@pytest.mark.parametrize("size", ODD, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_h_out_that_is_no_multiple_of_16(torch, size, dtype):
    """Beside the last codes of dy lie zeros, whatever the workspace held."""
    T, share, E, K, N = size
    torch.full((1 << 26,), 0x7f, dtype=torch.uint8, device="cuda")  # what an allocation may get next: NaN
    check(torch, T, share, E, K, N, dtype, seed=N, grouped=E > 1, pad=8)
    check(torch, T, share, E, K, N, dtype, seed=N, grouped=E > 1, narrow=True)


GROUPED = [(1, 2, 8, 512, 272), (5, 1, 3, 144, 400), (32, 2, 64, 272, 144), (40, 4, 5, 656, 528), (200, 2, 4, 1040, 272),
           (777, 1, 4, 272, 528), (7, 3, 1000, 144, 16), (500, 2, 9, 400, 656), (1500, 1, 2, 144, 1040)]


@pytest.mark.parametrize("size", GROUPED, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pad", [0, 40])
def test_grouped(torch, size, dtype, pad):
    T, share, E, K, N = size
    check(torch, T, share, E, K, N, dtype, seed=E, pad=pad)
    check(torch, T, share, E, K, N, dtype, seed=E, pad=pad, narrow=True)


@pytest.mark.parametrize("dx,size,form", list(block_sizes.cases()), ids=lambda v: str(v))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_every_form(torch, dx, size, form, dtype):
    """Each kernel form at sizes that test_block_forms.py checks to take it."""
    T, share, E, depth, out = size
    K, N = (out, depth) if dx else (depth, out)
    rows_of, share = (T * share, 1) if dx else (T, share)
    for narrow in (True, False):
        check(torch, rows_of, share, max(E, 1), K, N, dtype, seed=T, pad=8 * narrow, grouped=E > 0, forward=not dx, dx=dx,
              narrow=narrow)


@pytest.mark.parametrize("ids", [[-1] * 40, [2] * 40, [0, 1, 2, 3] * 10, [5] + [-1] * 38 + [0], [3] * 39 + [7]], ids=str)
def test_who_is_where(torch, ids):
    """No row of any group, one group alone, groups of one row."""
    for n in (40, 320):
        check(torch, n, 1, 4, 272, 144, "bf16", ids=(ids * 8)[:n])
        check(torch, n, 1, 4, 272, 144, "f16", ids=(ids * 8)[:n], narrow=True)


def test_every_column_and_block(torch):
    """One row of ones against a weight whose elements tell where they are: each block has a scale of its own."""
    import adapter_gemv_amd as sgmv
    K, N = 400, 656
    for T in (1, 40, 300, 3000, 9000):
        for at in (0, 127, 128, 200, 384, 399):
            x = torch.zeros(T, K, dtype=torch.bfloat16, device="cuda")
            x[:, at] = 1.0
            codes = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
            scales = torch.arange(1, 6 * 4 + 1, device="cuda", dtype=torch.float32).view(6, 4)
            y = sgmv.fp8_matmul(torch.empty(T, N, dtype=x.dtype, device="cuda"), x, sgmv.Fp8Weight(codes, scales))
            want = scales[torch.arange(N, device="cuda") // 128, at // 128].to(y.dtype)
            assert torch.equal(y, want.expand(T, N))
        for at in (0, 127, 128, 400, 640, 655):
            dy = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
            dy[:, at] = 1.0
            dx = sgmv.fp8_matmul_dx(torch.empty(T, K, dtype=x.dtype, device="cuda"), dy, sgmv.Fp8Weight(codes, scales))
            assert torch.equal(dx, scales[at // 128, torch.arange(K, device="cuda") // 128].to(dx.dtype).expand(T, K))


@pytest.mark.parametrize("T", [3, 40, 300, 3000, 9000])
def test_what_is_not_finite_stays_where_it_is(torch, T):
    """NaN codes, NaN and infinite scales, and rows that hold an infinity: their rows and columns, and no others."""
    import adapter_gemv_amd as sgmv
    K, N = 400, 272
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    W = weight(torch, gen, 1, N, K)
    clean = sgmv.Fp8Weight(W.codes.clone(), W.scales.clone())
    W.codes.view(torch.uint8)[0, 20, 399] = 0x7f
    W.codes.view(torch.uint8)[0, 150, 0] = 0xff
    x, dy = rows(torch, gen, T, K, "bf16", 0), rows(torch, gen, T, N, "bf16", 0)
    run = lambda x, W: sgmv.fp8_matmul(torch.empty(T, N, dtype=x.dtype, device="cuda"), x, W)  # noqa: E731
    run_dx = lambda d, W: sgmv.fp8_matmul_dx(torch.empty(T, K, dtype=d.dtype, device="cuda"), d, W)  # noqa: E731
    y0, d0, y, d = run(x, clean), run_dx(dy, clean), run(x, W), run_dx(dy, W)
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[[20, 150]] = False
    assert torch.isnan(y[:, ~keep]).all() and torch.equal(y[:, keep], y0[:, keep])
    keep = torch.ones(K, dtype=torch.bool, device="cuda")
    keep[[0, 399]] = False
    assert torch.isnan(d[:, ~keep]).all() and torch.equal(d[:, keep], d0[:, keep])
    # a row with an infinity
    x[T // 2, 399], dy[T // 2, 271] = float("inf"), float("nan")
    y, d = run(x, clean), run_dx(dy, clean)
    keep = torch.arange(T, device="cuda") != T // 2
    assert torch.isnan(y[T // 2]).all() and torch.equal(y[keep], y0[keep])
    assert torch.isnan(d[T // 2]).all() and torch.equal(d[keep], d0[keep])
    # a scale that is none: its block of columns
    clean.scales[0, 1, 3] = float("nan")
    x[T // 2, 399] = 0.0
    dy[T // 2, 271] = 0.0
    y, d = run(x, clean), run_dx(dy, clean)
    assert torch.isnan(y[:, 128:256]).all() and torch.equal(y[keep, :128], y0[keep, :128])
    assert torch.equal(y[keep, 256:], y0[keep, 256:]) and torch.isnan(d[:, 384:]).all()
    assert torch.equal(d[keep, :384], d0[keep, :384])


def test_scales_of_every_size(torch):
    """Products of scales from 2^-120 to 2^120: no step on the way passes float32's range."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    K, N = 272, 144
    for T in (4, 300):
        for power in (-110, -60, 0, 60, 100):
            W = weight(torch, gen, 1, N, K)
            W.scales.mul_(2.0 ** -power)
            x = rows(torch, gen, T, K, "bf16", 0) * 2.0 ** power
            Wd = np.stack([B.decode(c, s, 128) for c, s in zip(codes_of(W.codes, torch), f64(W.scales))])
            ref, mag = G.group_matmul(B.decode(*B.encode(f64(x), 1), 1), Wd, np.zeros(T, int))
            close(f64(sgmv.fp8_matmul(torch.empty(T, N, dtype=x.dtype, device="cuda"), x, W)), ref, mag, K, "bf16", f"2^{power}")


def test_past_32_bits(torch):
    """Rows that end past 2^32 bytes from their base, and codes of a group that start past them."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    K, N, E = 4096, 16384, 66
    W = sgmv.Fp8Weight(torch.zeros(E, N, K, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
                       torch.ones(E, N // 128, K // 128, device="cuda"))
    last = weight(torch, gen, 1, N, K)
    W.codes.view(torch.uint8)[E - 1].copy_(last.codes.view(torch.uint8)[0])
    W.scales[E - 1].copy_(last.scales[0])
    for T in (3, 200):
        ld = ((1 << 31) + (1 << 26)) // (T - 1) // 8 * 8
        near_x = rows(torch, gen, T, K, "bf16", 0).contiguous()
        store = torch.zeros((T - 1) * ld + N, dtype=torch.bfloat16, device="cuda")
        x = store.as_strided((T, K), (ld, 1))
        x.copy_(near_x)
        out = torch.zeros_like(store)
        y = out.as_strided((T, N), (ld, 1))
        groups = sgmv.group_rows(torch.full((T,), E - 1, dtype=torch.int32, device="cuda"), E)
        sgmv.fp8_matmul(y, x, W, groups)
        want = sgmv.fp8_matmul(torch.empty(T, N, dtype=y.dtype, device="cuda"), near_x, last)
        ref, mag = G.group_matmul(B.decode(*B.encode(f64(near_x), 1), 1),
                                  B.decode(codes_of(last.codes, torch)[0], f64(last.scales)[0], 128)[None], np.zeros(T, int))
        close(f64(want), ref, mag, K, "bf16", f"{T} rows")
        close(f64(y), ref, mag, K, "bf16", f"{T} rows far apart")
        dx = store.as_strided((T, K), (ld, 1))
        sgmv.fp8_matmul_dx(dx, y, W, groups)
        near = sgmv.fp8_matmul_dx(torch.empty(T, K, dtype=y.dtype, device="cuda"), y.contiguous(), last)
        ref, mag = G.group_matmul_dx(B.decode(*B.encode(f64(y), 1), 1),
                                     B.decode(codes_of(last.codes, torch)[0], f64(last.scales)[0], 128)[None], np.zeros(T, int))
        close(f64(near), ref, mag, N, "bf16", f"{T} rows dx")
        close(f64(dx), ref, mag, N, "bf16", f"{T} rows dx far apart")
        del store, out, x, y, dx


def test_untouched_rows_and_columns(torch):
    """What lies behind the output's columns stays."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for T in (2, 50, 300):
        W = weight(torch, gen, 1, 144, 272)
        store = torch.full((T + 2, 400), 7.0, dtype=torch.float16, device="cuda")
        sgmv.fp8_matmul(store[1:T + 1, 8:152], rows(torch, gen, T, 272, "f16", 8), W)
        assert bool((store[0] == 7).all()) and bool((store[T + 1] == 7).all()) and bool((store[:, :8] == 7).all())
        assert bool((store[:, 152:] == 7).all()) and not bool((store[1:T + 1, 8:152] == 7).all())
        store.fill_(7.0)
        sgmv.fp8_matmul_dx(store[1:T + 1, 8:280], rows(torch, gen, T, 144, "f16", 8), W)
        assert bool((store[0] == 7).all()) and bool((store[T + 1] == 7).all()) and bool((store[:, :8] == 7).all())
        assert bool((store[:, 280:] == 7).all())


def test_repeats_and_streams(torch):
    """The same bits each time, and on a stream of its own."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for T in (20, 700):
        W, x, dy = weight(torch, gen, 3, 400, 1040), rows(torch, gen, T, 1040, "bf16", 0), rows(torch, gen, T, 400, "bf16", 0)
        ids = torch.randint(0, 3, (T,), generator=gen, device="cuda", dtype=torch.int32)
        groups = sgmv.group_rows(ids, 3)
        y0 = sgmv.fp8_matmul(torch.empty_like(dy), x, W, groups)
        d0 = sgmv.fp8_matmul_dx(torch.empty_like(x), dy, W, groups)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        for stream in (None, None, s):
            y = sgmv.fp8_matmul(torch.empty_like(dy), x, W, groups, stream=stream)
            d = sgmv.fp8_matmul_dx(torch.empty_like(x), dy, W, groups, stream=stream)
            q = sgmv.fp8_quantize(x, stream=stream)
            qw = sgmv.fp8_quantize_weight(x[:16], stream=stream)
            back = sgmv.fp8_dequantize(torch.empty_like(x), q, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(y, y0) and torch.equal(d, d0) and back.isfinite().all() and qw.scales.isfinite().all()


def test_no_rows(torch):
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    W = weight(torch, gen, 3, 16, 32)
    x, y = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    groups = sgmv.group_rows(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert sgmv.fp8_matmul(y, x, W, groups) is y and sgmv.fp8_matmul_dx(x, y, W, groups) is x
    assert sgmv.fp8_quantize(x).shape == (0, 32)
