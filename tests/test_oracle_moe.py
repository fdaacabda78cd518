"""Pins of the routing oracle: closed forms, masks, groups, and the gradient against differences."""
import math

import numpy as np
import pytest

from oracle import moe


def test_closed_forms():
    ids, w = moe.route([[0.0, math.log(3), math.log(2)]], 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[0.6, 0.4]], rtol=1e-15)
    ids, w = moe.route([[0.0, math.log(3), math.log(2)]], 2, renormalize=False, scale=6.0)
    assert np.allclose(w, [[3.0, 2.0]], rtol=1e-15)
    ids, w = moe.route([[0.0, 0.0, 0.0]], 2, score="sigmoid", renormalize=False)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[0.5, 0.5]]
    ids, w = moe.route([[0.0, 0.0, 0.0]], 1, score="sigmoid", bias=[0, 0, 0.1])
    assert ids.tolist() == [[2]] and w.tolist() == [[1.0]]


def test_masks_and_wrong_rows():
    inf = math.inf
    ids, w = moe.route([[-inf, 1, -inf], [-inf] * 3, [1, inf, 0], [1, math.nan, 0]], 2)
    assert ids.tolist() == [[1, -1], [-1, -1], [0, 1], [0, 1]]
    assert w[0].tolist() == [1, 0] and w[1].tolist() == [0, 0] and np.isnan(w[2:]).all()
    ids, w = moe.route([[1, inf, -inf]], 2, score="sigmoid", renormalize=False)
    assert ids.tolist() == [[1, 0]] and w[0, 0] == 1


def test_groups():
    l = [[5.0, -9, 2, 2, 3, 0]]
    assert moe.route(l, 2, score="sigmoid", groups=3, top_groups=1)[0].tolist() == [[2, 3]]
    assert moe.route(l, 2, score="sigmoid", groups=3, top_groups=3)[0].tolist() == [[0, 4]]
    assert moe.route([[1.0] * 6], 2, groups=3, top_groups=1)[0].tolist() == [[0, 1]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(0)
    l, d = rng.standard_normal((5, 7)) * 2, rng.standard_normal((5, 3))
    l[1, 2] = l[2, :] = -math.inf
    how = dict(score=score, renormalize=renormalize, scale=1.7)
    ids, w = moe.route(l, 3, **how)
    assert np.allclose(w, moe.weights_at(l, ids, **how), rtol=1e-14)
    grad = moe.route_backward(l, ids, d, **how)
    h = 1e-5
    for t in range(5):
        for e in range(7):
            if l[t, e] == -math.inf:
                assert grad[t, e] == 0
                continue
            up, down = l.copy(), l.copy()
            up[t, e] += h
            down[t, e] -= h
            diff = ((moe.weights_at(up, ids, **how) - moe.weights_at(down, ids, **how)) * d).sum() / (2 * h)
            # (third derivatives of these functions are below 10: h^2 / 6 of them, and 2^-52 / h of the values)
            assert abs(diff - grad[t, e]) <= 1e-8


def test_group():
    off, rows, slots = moe.group([[2, 0], [9, 2], [-1, 0]], 3)
    assert off.tolist() == [0, 2, 2, 4] and rows.tolist() == [0, 2, 0, 1] and slots.tolist() == [[2, 0], [-1, 3], [-1, 1]]
