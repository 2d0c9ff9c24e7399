"""The weighted sum of each token's expert rows and its gradients against the fp64 oracle.

Tolerance: an output's own rounding (half a step) and, for each of the terms that it sums, two
float32 roundings of at most the sum of the magnitudes."""
import numpy as np
import pytest

from oracle import routing_oracle as R

pytestmark = pytest.mark.gpu
HALF = {"f16": (2.0 ** -11, 2.0 ** -25), "bf16": (2.0 ** -8, 2.0 ** -134)}


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def f64(t):
    return t.double().cpu().numpy()


def near(got, ref, tol, what):
    err = np.abs(got - ref)
    print(f"{what}: worst err/tol {(err / tol).max() if err.size else 0:.3f}", flush=True)
    assert np.all(err <= tol), f"{what}: {int((err > tol).sum())} of {err.size} outside"


def rows(torch, gen, n, h, t, pad):
    store = torch.full((n, h + pad), float("nan"), dtype=t, device="cuda")
    store[:, :h] = torch.randn(n, h, generator=gen, device="cuda").to(t)
    return store[:, :h]


SIZES = [(1, 1, 8), (1, 2, 4096), (3, 5, 264), (32, 2, 4096), (17, 8, 520), (64, 1, 2048), (5, 64, 2056),
         (300, 4, 136), (9, 3, 14336), (2000, 6, 1032), (2, 4, 40008), (3, 7, 72), (130, 16, 256)]


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("pad", [0, 24])
def test_sizes(torch, size, dtype, pad):
    import adapter_gemv_amd as sgmv
    T, k, h = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(T + h)
    t = torch.float16 if dtype == "f16" else torch.bfloat16
    u, sub = HALF[dtype]
    y, dout, out, dy = (rows(torch, gen, n, h, t, pad) for n in (T * k, T, T, T * k))
    w = torch.randn(T, k, generator=gen, device="cuda")
    w[0, 0] = 0.0
    Y, D, W, O = f64(y), f64(dout), f64(w), f64(out)
    for weights, Wn in ((w, W), (None, None)):
        ref, mag = R.combine(Y, Wn, k)
        held = out.clone()
        got = sgmv.combine_rows(torch.empty_like(out), y, weights)
        near(f64(got), ref, u * np.abs(ref) + sub + 2 * (k + 1) * 2.0 ** -24 * mag, f"{size} {dtype}")
        got = sgmv.combine_rows(out, y, weights, add=True)
        assert got is out
        near(f64(out), ref + O, u * np.abs(ref + O) + sub + 2 * (k + 2) * 2.0 ** -24 * (mag + np.abs(O)), f"{size} {dtype} add")
        out.copy_(held)
    dw = torch.full((T, k), float("nan"), device="cuda")
    got = sgmv.combine_rows_backward(dy, dw, dout, y, w)
    assert got[0] is dy and got[1] is dw
    rdy, rdw, mag = R.combine_backward(D, Y, W, k)
    near(f64(dy), rdy, u * np.abs(rdy) + sub + 2.0 ** -24 * np.abs(rdy), f"{size} {dtype} dy")
    near(f64(dw), rdw, 2.0 ** -24 * (h + 8) * mag + 2.0 ** -140, f"{size} {dtype} dw")
    sgmv.combine_rows_backward(dy, None, dout)
    assert torch.equal(dy, dout.repeat_interleave(k, 0))


def test_past_32_bits(torch):
    """Rows that end past 2^32 bytes from their base."""
    import adapter_gemv_amd as sgmv
    T, k, h = 3, 2, 72
    ld = (1 << 30) // 8 * 8
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    t = torch.bfloat16
    big, other = (torch.zeros(5 * ld + 1024, dtype=t, device="cuda") for _ in range(2))
    y, dy = big.as_strided((6, h), (ld, 1)), other.as_strided((6, h), (ld, 1))
    y.copy_(torch.randn(6, h, generator=gen, device="cuda"))
    w = torch.randn(T, k, generator=gen, device="cuda")
    near_y = y.contiguous()
    assert torch.equal(sgmv.combine_rows(torch.empty(T, h, dtype=t, device="cuda"), y, w),
                       sgmv.combine_rows(torch.empty(T, h, dtype=t, device="cuda"), near_y, w))
    dout = torch.randn(T, h, generator=gen, device="cuda").to(t)
    dw, dw1 = torch.empty_like(w), torch.empty_like(w)
    sgmv.combine_rows_backward(dy, dw, dout, y, w)
    dy1, _ = sgmv.combine_rows_backward(torch.empty_like(near_y), dw1, dout, near_y, w)
    assert torch.equal(dy, dy1) and torch.equal(dw, dw1)


def test_what_is_not_finite_stays_in_its_token(torch):
    import adapter_gemv_amd as sgmv
    y = torch.ones(12, 520, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(6, 2, device="cuda")
    y[3, 7], y[8, 9], w[5, 1] = float("nan"), float("inf"), float("inf")
    out = sgmv.combine_rows(torch.empty(6, 520, dtype=y.dtype, device="cuda"), y, w)
    bad = ~torch.isfinite(out)
    assert bad[1].nonzero().flatten().tolist() == [7] and bad[4].nonzero().flatten().tolist() == [9]
    assert bool(bad[5].all()) and not bool(bad[[0, 2, 3]].any())
    dw = torch.empty_like(w)
    sgmv.combine_rows_backward(torch.empty_like(y), dw, torch.ones_like(out), y, w)
    assert (~torch.isfinite(dw)).nonzero().tolist() == [[1, 1], [4, 0]]


def test_no_tokens_and_streams(torch):
    import adapter_gemv_amd as sgmv
    e = torch.empty(0, 64, dtype=torch.float16, device="cuda")
    w = torch.empty(0, 3, device="cuda")
    assert sgmv.combine_rows(e, e, w) is e and sgmv.combine_rows(e, e) is e
    sgmv.combine_rows_backward(e, w, e, e, w)
    y = torch.randn(40, 64, device="cuda").half()
    w = torch.randn(10, 4, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = sgmv.combine_rows(torch.empty(10, 64, dtype=y.dtype, device="cuda"), y, w, stream=s)
    s.synchronize()
    assert torch.equal(a, sgmv.combine_rows(torch.empty_like(a), y, w))


def test_gradient_against_differences(torch):
    """The sum is linear in the rows and in the weights: sums of steps of one are exact quotients (small whole
    numbers, which float16 holds)."""
    import adapter_gemv_amd as sgmv
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    y = torch.randint(-3, 4, (6, 16), generator=gen, device="cuda").half()
    w = torch.randint(-3, 4, (2, 3), generator=gen, device="cuda").float()
    g = torch.randint(-3, 4, (2, 16), generator=gen, device="cuda").half()
    dw = torch.empty_like(w)
    dy, _ = sgmv.combine_rows_backward(torch.empty_like(y), dw, g, y, w)
    total = lambda y, w: float((sgmv.combine_rows(torch.empty_like(g), y, w).double() * g.double()).sum())  # noqa: E731
    base = total(y, w)
    for i in range(6):
        for c in (0, 7, 15):
            y1 = y.clone()
            y1[i, c] += 1
            assert total(y1, w) - base == float(dy[i, c])
        w1 = w.clone()
        w1.view(-1)[i] += 1
        assert total(y, w1) - base == float(dw.view(-1)[i])
