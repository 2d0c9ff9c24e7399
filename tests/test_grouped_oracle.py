"""The fp64 definitions of the grouped products and of the 4-bit format, pinned by worked
examples and by the formula element by element."""
import numpy as np
import pytest

from oracle import grouped_oracle as G


def test_group_rows_worked_example():
    starts, perm = G.group_rows([2, -1, 0, 2, 5, 0], 3)
    assert perm.tolist() == [2, 5, 0, 3, 1, 4]      # groups 0, 2, then the two of no group
    assert starts.tolist() == [0, 2, 2, 4]


def test_products_element_by_element():
    rng = np.random.default_rng(5)
    n, share, E, K, N = 6, 2, 3, 4, 5
    x, W = rng.standard_normal((n // share, K)), rng.standard_normal((E, N, K))
    dy, ids = rng.standard_normal((n, N)), np.array([0, 2, 2, -1, 0, 7])
    y, _ = G.group_matmul(x, W, ids, share)
    dx, _ = G.group_matmul_dx(dy, W, ids)
    dW, _ = G.group_matmul_dw(x, dy, ids, E, share)
    y2, dx2, dW2 = np.zeros_like(y), np.zeros_like(dx), np.zeros_like(dW)
    for i, g in enumerate(ids):
        if 0 <= g < E:
            for o in range(N):
                for k in range(K):
                    y2[i, o] += x[i // share, k] * W[g, o, k]
                    dx2[i, k] += dy[i, o] * W[g, o, k]
                    dW2[g, o, k] += dy[i, o] * x[i // share, k]
    for a, b in ((y, y2), (dx, dx2), (dW, dW2)):
        assert np.allclose(a, b, rtol=0, atol=1e-12)


def test_mx_worked_block():
    v = np.zeros(32)
    v[:10] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.0, -5.1]   # top 7.9: scale 1
    codes, scales = G.mx_encode(v)
    assert scales.tolist() == [127]
    assert G.mx_decode(codes, scales)[:10].tolist() == [0, 1, 1, 2, 2, 4, 4, 6, 0, -6]
    assert codes[0] == 0 + 16 * 2 and codes[4] == 8 + 16 * 15        # low half: the even place


@pytest.mark.parametrize("top,scale", [(1.0, 125), (8.0, 128), (7.99, 127), (2.0 ** -130, 0),
                                       (0.0, 0), (np.inf, 255), (np.nan, 255)])
def test_mx_scale(top, scale):
    v = np.full(64, 1.0)
    v[32:] = 0.0
    v[40] = top
    codes, scales = G.mx_encode(v)
    assert scales.tolist() == [125, scale]
    back = G.mx_decode(codes, scales)
    assert np.array_equal(back[:32], np.ones(32))
    assert np.isnan(back[32:]).all() == (scale == 255)
