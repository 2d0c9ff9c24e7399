"""The oracles of routing and of 8-bit blocks against worked examples, closed forms and
differences."""
import math

import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import routing_oracle as R


def test_worked_example():
    # two groups of three; scores softmax of log(1, 2, 3 | 4, 4, 2) = the same over 16
    row = [math.log(v) for v in (1, 2, 3, 4, 4, 2)]
    assert R.choose(row, 3) == [3, 4, 2]
    # group sums of two: 5 and 8; of one: 3 and 4; a bias may turn them round, and order experts
    assert R.choose(row, 3, groups=2, keep=1) == [3, 4, 5]
    assert R.choose(row, 3, groups=2, keep=1, bias=[0, 0, 0.25, 0, 0, 0]) == [2, 1, 0]
    assert R.choose(row, 2, bias=[1, 0, 0, 0, 0, 0]) == [0, 3]
    ids, w = R.route([row], 2, normalize=False, scale=2.0)
    assert np.allclose(w, [[0.5, 0.5]]) and ids.tolist() == [[3, 4]]
    ids, w = R.route([row], 3)
    assert np.allclose(w, [[4 / 11, 4 / 11, 3 / 11]])
    ids, w = R.route([row], 3, scores="sigmoid", normalize=False)   # v / (1 + v)
    assert np.allclose(w, [[4 / 5, 4 / 5, 3 / 4]])


def test_masks_and_what_is_no_number():
    inf = math.inf
    ids, w = R.route([[-inf] * 4, [-inf, 1.0, -inf, -inf], [0.0, math.nan, 1.0, -inf]], 2)
    assert ids.tolist() == [[-1, -1], [1, -1], [0, 1]]
    assert w[0].tolist() == [0, 0] and w[1].tolist() == [1, 0] and np.isnan(w[2]).all()
    ids, w = R.route([[0.0, math.nan, 1.0, 2.0]], 2, scores="sigmoid", normalize=False)
    assert ids.tolist() == [[1, 3]] and np.isnan(w[0, 0]) and w[0, 1] == 1 / (1 + math.exp(-2))
    # a group without experts never stays, one with a single expert counts it alone
    row = [-inf, -inf, 0.0, -inf, -5.0, -6.0]
    assert R.choose(row, 6, groups=3, keep=2, scores="sigmoid") == [2, 4, 5]
    assert R.choose(row, 6, groups=3, keep=3) == [2, 4, 5]


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_gradient_against_differences(scores, normalize):
    rng = np.random.default_rng(3)
    l, g = rng.normal(size=(5, 9)), rng.normal(size=(5, 4))
    l[0, 3] = -math.inf
    ids, _ = R.route(l, 4, scores=scores)
    d, _ = R.route_backward(l, ids, g, scores, normalize, 1.5)
    h = 1e-6
    for t in range(5):
        for i in range(9):
            if l[t, i] == -math.inf:
                assert d[t, i] == 0
                continue
            f = []
            for step in (h, -h):
                row = list(l[t])
                row[i] += step
                f.append(1.5 * np.dot(g[t], R.shares(row, list(ids[t]), scores, normalize)))
            assert abs((f[0] - f[1]) / (2 * h) - d[t, i]) < 1e-8


def test_combine_against_differences():
    rng = np.random.default_rng(4)
    y, w, g = rng.normal(size=(6, 5)), rng.normal(size=(3, 2)), rng.normal(size=(3, 5))
    out, _ = R.combine(y, w, 2)
    assert np.allclose(out[1], w[1, 0] * y[2] + w[1, 1] * y[3])
    dy, dw, _ = R.combine_backward(g, y, w, 2)
    # the sum is linear in each: a step of one gives the gradient
    for i in range(6):
        step = np.zeros_like(y)
        step[i, 2] = 1.0
        assert np.isclose(((R.combine(y + step, w, 2)[0] - out) * g).sum(), dy[i, 2])
    step = np.zeros_like(w)
    step[2, 1] = 1.0
    assert np.isclose(((R.combine(y, w + step, 2)[0] - out) * g).sum(), dw[2, 1])
    assert np.array_equal(R.combine(y, None, 2)[0], y[0::2] + y[1::2])


def test_eight_bit_values():
    assert B.VALUES[0x7e] == 448 and B.VALUES[1] == 2.0 ** -9 and B.VALUES[0x38] == 1 and B.VALUES[0x08] == 2.0 ** -6
    assert np.isnan(B.VALUES[[0x7f, 0xff]]).all() and np.isfinite(np.delete(B.VALUES, [0x7f, 0xff])).all()
    codes = np.array([c for c in range(256) if c & 0x7f != 0x7f], np.uint8)
    assert np.array_equal(B.nearest(B.VALUES[codes]), codes)
    # halfway between neighbours: the even code
    sizes = B.VALUES[:127]
    mid = (sizes[:-1] + sizes[1:]) / 2
    got = B.nearest(mid)
    assert np.all(got % 2 == 0) and np.all((got == np.arange(126)) | (got == np.arange(1, 127)))
    assert np.array_equal(B.nearest(mid * (1 + 1e-9)), np.arange(1, 127))
    assert np.array_equal(B.nearest(-mid * (1 - 1e-9)), np.arange(126) + 128)


def test_eight_bit_scales():
    for top, want in ((448.0, 1.0), (448.1, 2.0), (1.75, 2.0 ** -8), (1.7500001, 2.0 ** -7), (1.0, 2.0 ** -8),
                      (0.0, 2.0 ** -126), (2.0 ** -130, 2.0 ** -126), (2.0 ** -118 * 1.75, 2.0 ** -126),
                      (2.0 ** -118 * 1.8, 2.0 ** -125), (3.38e38, 2.0 ** 120)):
        assert B.scale_of(top) == want, top
    v = np.zeros((3, 144))
    v[0, 0], v[1, 130], v[2, 5] = 3.0, -448.0, math.inf
    codes, s = B.encode(v, 1)
    assert s.shape == (3, 2) and s[0, 0] == 2.0 ** -7 and s[1, 1] == 1 and np.isnan(s[2, 0]) and s[2, 1] == 2.0 ** -126
    assert B.decode(codes, s, 1)[0, 0] == 3.0 and B.decode(codes, s, 1)[1, 130] == -448 and not codes[2].any()
    codes, s = B.encode(v[:2], 128)
    assert s.shape == (1, 2) and s[0].tolist() == [2.0 ** -7, 1.0]
