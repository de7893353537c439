"""Float64 definitions of the operators around the expert layer in a training
step (test infrastructure only): layer norm, softmax cross entropy over a
vocabulary, the global gradient norm and clipping.  Plain numpy, written from
the formulas; nothing here is shared with the CUDA path."""
from __future__ import annotations

import numpy as np


def layer_norm(x, gamma, beta, eps):
    """(y, mean, rstd) of rows x [T, H]; gamma / beta None: 1 / 0."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, gamma, eps):
    """(dx, dgamma, dbeta)."""
    dy = np.asarray(dy, np.float64)
    x = np.asarray(x, np.float64)
    h, _, rstd = layer_norm(x, None, None, eps)
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = rstd[:, None] * (g - g.mean(1)[:, None] - h * (g * h).mean(1)[:, None])
    return dx, (dy * h).sum(0), dy.sum(0)


def counted(targets, V, ignore):
    """Which rows count: the target is in the vocabulary and not ignored."""
    t = np.asarray(targets, np.int64)
    return (t != ignore) & (t >= 0) & (t < V)


def cross_entropy(X, W, targets, ignore=-100):
    """(loss [T], lse [T], mean over the rows that count)."""
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    t = np.asarray(targets, np.int64)
    z = X @ W.T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    on = counted(t, W.shape[0], ignore)
    loss = np.zeros(len(t))
    rows = np.nonzero(on)[0]
    loss[rows] = lse[rows] - z[rows, t[rows]]
    return loss, lse, (loss.sum() / on.sum() if on.any() else 0.0)


def cross_entropy_backward(X, W, targets, dloss, ignore=-100):
    """(dX, dW, dz) with dloss [T] the gradient that reaches each row's loss."""
    X, W = np.asarray(X, np.float64), np.asarray(W, np.float64)
    t = np.asarray(targets, np.int64)
    _, lse, _ = cross_entropy(X, W, t, ignore)
    on = counted(t, W.shape[0], ignore)
    dz = np.exp(X @ W.T - lse[:, None])
    rows = np.nonzero(on)[0]
    dz[rows, t[rows]] -= 1.0
    dz[~on] = 0.0
    dz[rows] *= np.asarray(dloss, np.float64)[rows][:, None]
    return dz @ W, dz.T @ X, dz


def grad_norm(tensors):
    """sqrt of the sum of all squares."""
    return float(np.sqrt(sum(float((np.asarray(t, np.float64) ** 2).sum()) for t in tensors)))


def clip_grads(tensors, max_norm):
    """(norm, scaled tensors)."""
    n = grad_norm(tensors)
    c = max_norm / n if n > max_norm else 1.0
    return n, [np.asarray(t, np.float64) * c for t in tensors]
