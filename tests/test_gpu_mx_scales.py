"""4-bit products whose scales take elements past what 16-bit types hold, in every form of the
kernels, against the fp64 oracle: results depend neither on the number of rows nor on which
other scales share a workgroup.  Tolerance: as in the grouped products' tests."""
import sys

import numpy as np
import pytest

from oracle import grouped_oracle as G

pytestmark = pytest.mark.gpu

# rows, h_in, h_out: the streaming kernels of 8 wavefronts and of 32 columns with 16 rows and with
# 32, then the tiled kernels of 128 x 128, 128 x 256 and 256 x 256; the last two are for the
# streaming kernels with both sides in 4 bits
SIZES = [(3, 2080, 264), (24, 2304, 264), (5, 2080, 8200), (24, 2304, 8200), (300, 160, 264),
         (1100, 160, 7000), (4096, 160, 4096), (24, 8416, 264), (5, 5152, 8200)]


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch


def close(got, ref, mag, depth, dtype, what):
    u, sub, most = (2.0 ** -8, 2.0 ** -134, 3.39e38) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25, 65504.0)
    tol = u * np.abs(ref) + sub + (1 + u) * (depth + 32) * 2.0 ** -23 * mag
    over = np.abs(ref) - tol > most * (1 + u)         # beyond the type: infinite, of its sign
    assert np.array_equal(got[over], np.copysign(np.inf, ref[over])), what
    near = ~over & (np.abs(ref) + tol >= most)        # either side
    ok = ~over & ~near
    err = np.abs(got[ok] - ref[ok])
    worst = (err / tol[ok]).max() if err.size else 0
    print(f"{what}: {ok.sum()} of {ok.size} finite, worst err/tol {worst:.3f}", flush=True)
    sys.stdout.flush()
    assert np.all(err <= tol[ok]), f"{what}: {int((err > tol[ok]).sum())} outside"


def random_codes(torch, gen, *shape):
    return torch.randint(0, 256, shape, generator=gen, device="cuda", dtype=torch.uint8)


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("low,high,power", [(245, 254, -118), (252, 252, -110), (0, 3, 118), (0, 254, -120)])
def test_scales_at_the_ends_of_the_range(torch, size, low, high, power):
    """Elements up to 6 * 2^127, which bfloat16 and float32 do not hold, times rows that bring
    the products back, and elements down to 2^-128."""
    import adapter_gemv_amd as sgmv
    rows, K, N = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(low + high)
    q = sgmv.MxTensor(random_codes(torch, gen, N, K // 2),
                      torch.randint(low, high + 1, (N, K // 32), generator=gen, device="cuda", dtype=torch.uint8))
    x = (torch.randn(rows, K, generator=gen, device="cuda") * 2.0 ** power).bfloat16()
    W = G.mx_decode(q.codes.cpu().numpy(), q.scales.cpu().numpy())[None]
    for both in (False, True):
        y = sgmv.mx_matmul(torch.full((rows, N), float("nan"), dtype=x.dtype, device="cuda"),
                           sgmv.mx_quantize(x) if both else x, q)
        X = x.double().cpu().numpy()
        X = G.mx_decode(*G.mx_encode(X)) if both else X
        for lo in range(0, rows, 512):
            ref, mag = G.group_matmul(X[lo:lo + 512], W, np.zeros(len(X[lo:lo + 512]), int))
            close(y[lo:lo + 512].double().cpu().numpy(), ref, mag, K, "bf16", f"{size} both {both} rows {lo}..")


@pytest.mark.parametrize("size", SIZES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_one_large_scale_spoils_nothing_else(torch, size, dtype):
    """Blocks scaled by 2^126 and 2^127 in the first, a middle and the last block of a row meet
    zeros in x: every product is ordinary, also beside the smallest scales and an infinity."""
    import adapter_gemv_amd as sgmv
    rows, K, N = size
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    t = torch.bfloat16 if dtype == "bf16" else torch.float16
    blocks = K // 32
    at = [0, blocks // 2, blocks - 1]
    scales = torch.randint(108, 135, (N, blocks), generator=gen, device="cuda", dtype=torch.uint8)
    scales[:, 1] = torch.randint(0, 4, (N,), generator=gen, device="cuda", dtype=torch.uint8)
    for i, b in enumerate(at):
        scales[i::7, b] = 253 + i % 2
    codes = random_codes(torch, gen, N, K // 2)
    x = torch.randn(rows, K, generator=gen, device="cuda").to(t)
    for b in at:
        x[:, 32 * b:32 * b + 32] = 0
    q = sgmv.MxTensor(codes, scales)
    W = G.mx_decode(codes.cpu().numpy(), scales.cpu().numpy())[None]
    for both in (False, True):
        X = x.double().cpu().numpy()
        X = G.mx_decode(*G.mx_encode(X)) if both else X
        y = sgmv.mx_matmul(torch.full((rows, N), float("nan"), dtype=t, device="cuda"),
                           sgmv.mx_quantize(x) if both else x, q)
        for lo in range(0, rows, 512):
            ref, mag = G.group_matmul(X[lo:lo + 512], W, np.zeros(len(X[lo:lo + 512]), int))
            close(y[lo:lo + 512].double().cpu().numpy(), ref, mag, K, dtype, f"{size} both {both} rows {lo}..")
    # an infinity in one row of x, where no weight of the columns is zero: infinite or NaN there, and
    # nowhere else
    x[rows // 2, 40] = float("inf")
    codes[:, 20] |= 0x11
    y2 = sgmv.mx_matmul(torch.empty(rows, N, dtype=t, device="cuda"), x, q)
    keep = torch.arange(rows, device="cuda") != rows // 2
    assert torch.isinf(y2[rows // 2]).all()
    x[rows // 2, 40] = 0
    y3 = sgmv.mx_matmul(torch.empty(rows, N, dtype=t, device="cuda"), x, q)
    assert torch.equal(y2[keep], y3[keep]) and torch.isfinite(y3).all()
