"""The float64 definitions of the training-step operators, pinned by central
differences, by invariants and by hand-worked cases (CPU)."""
import numpy as np
import pytest

from oracle import training_oracle as O

H_STEP = 1e-5      # central differences in float64: truncation ~h^2, rounding ~1e-16/h


def _diff(f, x, d):
    """Derivative of the number f(x) along d."""
    return (f(x + H_STEP * d) - f(x - H_STEP * d)) / (2 * H_STEP)


@pytest.mark.parametrize("T,H", [(1, 1), (3, 5), (4, 16)])
def test_layer_norm_gradients_are_the_differences(T, H):
    rng = np.random.default_rng(T * 10 + H)
    x, dy = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    g, b = 1 + 0.3 * rng.standard_normal(H), rng.standard_normal(H)
    eps = 1e-2
    dx, dg, db = O.layer_norm_backward(dy, x, g, eps)
    d = rng.standard_normal((T, H))
    e = rng.standard_normal(H)
    assert np.isclose((dx * d).sum(), _diff(lambda v: (O.layer_norm(v, g, b, eps)[0] * dy).sum(), x, d),
                      rtol=1e-7, atol=1e-8)
    assert np.isclose(dg @ e, _diff(lambda v: (O.layer_norm(x, v, b, eps)[0] * dy).sum(), g, e),
                      rtol=1e-7, atol=1e-8)
    assert np.isclose(db @ e, _diff(lambda v: (O.layer_norm(x, g, v, eps)[0] * dy).sum(), b, e),
                      rtol=1e-7, atol=1e-8)


def test_layer_norm_invariants():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 64))
    y, mean, rstd = O.layer_norm(x, None, None, 0.0)
    assert np.allclose(y.mean(1), 0) and np.allclose((y * y).mean(1), 1)
    assert np.allclose(O.layer_norm(3 * x + 7, None, None, 0.0)[0], y)
    dx, _, _ = O.layer_norm_backward(rng.standard_normal((5, 64)), x, None, 0.0)
    assert np.allclose(dx.sum(1), 0) and np.allclose((dx * y).sum(1), 0)


def test_cross_entropy_gradients_are_the_differences():
    rng = np.random.default_rng(1)
    X, W = rng.standard_normal((6, 8)), rng.standard_normal((11, 8))
    t = np.array([0, 10, 3, -100, 5, 99])        # one ignored, one outside the vocabulary
    s = rng.standard_normal(6)
    dX, dW, dz = O.cross_entropy_backward(X, W, t, s)
    D, E = rng.standard_normal(X.shape), rng.standard_normal(W.shape)
    assert np.isclose((dX * D).sum(), _diff(lambda v: (O.cross_entropy(v, W, t)[0] * s).sum(), X, D),
                      rtol=1e-7, atol=1e-8)
    assert np.isclose((dW * E).sum(), _diff(lambda v: (O.cross_entropy(X, v, t)[0] * s).sum(), W, E),
                      rtol=1e-7, atol=1e-8)
    assert not dz[3].any() and not dz[5].any() and np.allclose(dz.sum(1), 0)


def test_cross_entropy_by_hand():
    X, W = np.array([[1.0, 0.0], [0.0, 2.0]]), np.array([[0.0, 0.0], [0.0, 0.0], [0.0, 0.0]])
    loss, lse, mean = O.cross_entropy(X, W, [2, -100])
    assert np.allclose(loss, [np.log(3), 0]) and np.allclose(lse, np.log(3)) and np.isclose(mean, np.log(3))
    assert O.cross_entropy(X, W, [-100, -100])[2] == 0.0
    assert np.allclose(O.cross_entropy(X, W[:1], [0, 0])[0], 0)     # one entry: no choice


def test_clipping_by_hand():
    t = [np.array([3.0]), np.array([[0.0, 4.0]])]
    n, out = O.clip_grads(t, 1.0)
    assert n == 5.0 and np.allclose(out[0], 0.6) and np.allclose(out[1], [[0, 0.8]])
    n, out = O.clip_grads(t, 7.0)
    assert n == 5.0 and out[0] == 3.0
