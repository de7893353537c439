"""The float64 definitions of routing by scores and of the RMS norm, pinned by
central differences, brute force and hand-worked cases (CPU)."""
import itertools

import numpy as np
import pytest

from oracle import moe_oracle as M
from oracle import training_oracle as O

H_STEP = 1e-5      # central differences in float64: truncation ~h^2, rounding ~1e-16/h


def _diff(f, x, d):
    return (f(x + H_STEP * d) - f(x - H_STEP * d)) / (2 * H_STEP)


@pytest.mark.parametrize("score,renorm", list(itertools.product(["softmax", "sigmoid"], [True, False])))
@pytest.mark.parametrize("groups", [1, 4])
def test_router_gradient_is_the_difference(score, renorm, groups):
    rng = np.random.default_rng(groups)
    l, b, dg = rng.standard_normal((5, 16)), 0.1 * rng.standard_normal(16), rng.standard_normal((5, 3))
    how = dict(score=score, groups=groups, top_groups=2 if groups > 1 else 1, group_top=2 if groups > 1 else 1,
               renormalise=renorm, scale=2.5)
    idx, gate = O.route_by_scores(l, b, 3, **how)

    def gates(v):
        i, g = O.route_by_scores(v, b, 3, **how)
        assert np.array_equal(i, idx)                # the choice does not change over the step
        return g
    dl = O.route_by_scores_backward(l, idx, gate, dg, score, renorm, 2.5)
    for _ in range(4):
        d = rng.standard_normal(l.shape)
        assert np.isclose((dl * d).sum(), _diff(lambda v: (gates(v) * dg).sum(), l, d), rtol=1e-7, atol=1e-8)


def test_router_without_extras_is_the_softmax_router():
    rng = np.random.default_rng(0)
    l = np.round(rng.standard_normal((40, 24)) * 4) / 4          # with ties
    l[3, 5:] = -np.inf
    idx, gate = O.route_by_scores(l, None, 6)
    want, g = M.route(l, 6)
    assert np.array_equal(idx, want) and np.allclose(gate, g)
    dg = rng.standard_normal((40, 6))
    assert np.allclose(O.route_by_scores_backward(l, idx, gate, dg), M.route_backward(gate, idx, dg, 24))


def test_router_by_hand():
    l = np.log(np.array([[1.0, 2.0, 3.0, 4.0]]))
    # softmax .1 .2 .3 .4; the bias moves expert 0 to the front, its gate stays that of its score
    idx, gate = O.route_by_scores(l, [1.0, 0, 0, 0], 2, renormalise=False, scale=2.0)
    assert idx.tolist() == [[0, 3]] and np.allclose(gate, [[0.2, 0.8]])
    # groups {0, 1} and {2, 3}, by their sums .3 and .7
    idx, gate = O.route_by_scores(l, None, 2, groups=2, top_groups=1, group_top=2)
    assert idx.tolist() == [[3, 2]] and np.allclose(gate, [[4 / 7, 3 / 7]])
    # by their largest: a group of one large and one masked expert
    l = np.array([[5.0, -np.inf, 1.0, 2.0]])
    assert O.route_by_scores(l, None, 2, groups=2, top_groups=1, group_top=1)[0].tolist() == [[0, 1]]
    assert O.route_by_scores(l, None, 2, groups=2, top_groups=1, group_top=2)[0].tolist() == [[3, 2]]
    # sigmoid: 1/2 and 3/4
    idx, gate = O.route_by_scores(np.array([[0.0, np.log(3.0)]]), None, 2, score="sigmoid", renormalise=False)
    assert idx.tolist() == [[1, 0]] and np.allclose(gate, [[0.75, 0.5]])
    # a masked expert is last whatever its bias; nothing but masked ones: gates 0
    idx, gate = O.route_by_scores(np.array([[-np.inf, 0.0, 1.0]] * 2), [9.0, 0, 0], 3, score="sigmoid")
    assert idx[0].tolist() == [2, 1, 0] and gate[0, 2] == 0
    idx, gate = O.route_by_scores(np.full((1, 4), -np.inf), None, 2)
    assert idx.tolist() == [[0, 1]] and not gate.any()


def test_balance_by_hand():
    assert np.allclose(O.balance_bias([4, 2, 3], 0.5, [0.0, 0, 1]), [-0.5, 0.5, 1])


@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (4, 16)])
def test_rms_gradients_are_the_differences(T, H):
    rng = np.random.default_rng(T * 10 + H)
    x, r, dy, dh = (rng.standard_normal((T, H)) for _ in range(4))
    g, eps = 1 + 0.3 * rng.standard_normal(H), 1e-2
    h, _, rstd = O.rms_norm(x, r, g, eps)
    dx, dg = O.rms_norm_backward(dy, h, g, rstd, dh)

    def f(x, r, g):
        h, y, _ = O.rms_norm(x, r, g, eps)
        return (y * dy).sum() + (h * dh).sum()
    d, e = rng.standard_normal((T, H)), rng.standard_normal(H)
    assert np.isclose((dx * d).sum(), _diff(lambda v: f(v, r, g), x, d), rtol=1e-7, atol=1e-8)
    assert np.isclose((dx * d).sum(), _diff(lambda v: f(x, v, g), r, d), rtol=1e-7, atol=1e-8)
    assert np.isclose(dg @ e, _diff(lambda v: f(x, r, v), g, e), rtol=1e-7, atol=1e-8)


def test_rms_by_hand():
    h, y, rstd = O.rms_norm([[1.0, 5.0]], [[2.0, -1.0]], [1.0, 2.0], 0.0)
    assert np.allclose(h, [[3, 4]]) and np.allclose(rstd, 1 / np.sqrt(12.5)) and np.allclose(y, [[3, 8]] * rstd)
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 64))
    h, y, rstd = O.rms_norm(x, None, None, 0.0)
    assert np.allclose((y * y).mean(1), 1) and np.allclose(O.rms_norm(3 * x, None, None, 0.0)[1], y)
    assert np.allclose((O.rms_norm_backward(rng.standard_normal((5, 64)), h, None, rstd)[0] * y).sum(1), 0)
