"""Float64 definitions of the operators around the expert layer in a training
step (test infrastructure only): routing by scores, layer norm, RMS norm, softmax
cross entropy over a vocabulary, the global gradient norm and clipping.  Plain numpy, written from
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


def _readable(logits):
    """NaN and +inf read as -inf (a masked expert)."""
    l = np.asarray(logits, np.float64)
    return np.where(np.isnan(l) | (l == np.inf), -np.inf, l)


def scores(logits, score):
    """s [T, E]; 0 for masked experts."""
    l = _readable(logits)
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    top = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def route_by_scores(logits, bias, k, score="softmax", groups=1, top_groups=1, group_top=1, renormalise=True,
                    scale=1.0):
    """(idx, gate) [T, k], by sorting with Python."""
    l = _readable(logits)
    T, E = l.shape
    size = E // groups
    s = scores(l, score)
    b = np.zeros(E) if bias is None else np.where(np.isfinite(bias), np.asarray(bias, np.float64), 0.0)
    by_logit = bias is None and (groups == 1 or group_top == 1)
    u = l if by_logit else np.where(np.isfinite(l), s + b, -np.inf)
    idx = np.zeros((T, k), np.int64)
    for t in range(T):
        value = [sum(sorted(u[t, g * size:(g + 1) * size])[::-1][:group_top]) for g in range(groups)]
        stay = sorted(range(groups), key=lambda g: (-value[g], g))[:top_groups]
        eligible = [e for e in range(E) if e // size in stay]
        idx[t] = sorted(eligible, key=lambda e: (-u[t, e], e))[:k]
    ls = np.take_along_axis(l, idx, 1)
    if renormalise:
        x = -np.logaddexp(0, -ls) if score == "sigmoid" else ls
        top = x.max(1, keepdims=True)
        w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        w = w / np.maximum(w.sum(1, keepdims=True), 1e-300)
    else:
        w = np.take_along_axis(s, idx, 1)
    return idx, scale * w


def route_by_scores_backward(logits, idx, gate, dgate, score="softmax", renormalise=True, scale=1.0):
    """dlogits [T, E] with the choice held fixed."""
    l, dg = _readable(logits), np.asarray(dgate, np.float64)
    inner = (gate * dg).sum(1, keepdims=True)
    out = np.zeros_like(l)
    d = gate * (dg - inner / scale) if renormalise else gate * dg
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            d = d / (1.0 + np.exp(np.take_along_axis(l, idx, 1)))
    elif not renormalise:
        out = -scores(l, score) * inner
    np.put_along_axis(out, idx, np.take_along_axis(out, idx, 1) + d, 1)
    return out


def balance_bias(counts, rate, bias):
    counts = np.asarray(counts, np.int64)
    return np.asarray(bias, np.float64) + rate * np.sign(counts.sum() - counts * len(counts))


def rms_norm(x, residual, gamma, eps):
    """(h, y, rstd)."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(1) + eps)
    y = h * rstd[:, None]
    return h, y if gamma is None else y * np.asarray(gamma, np.float64), rstd


def rms_norm_backward(dy, h, gamma, rstd, dh=None):
    """(dx, dgamma)."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    xh = h * np.asarray(rstd, np.float64)[:, None]
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = np.asarray(rstd)[:, None] * (g - xh * (g * xh).mean(1)[:, None])
    return dx if dh is None else dx + np.asarray(dh, np.float64), (dy * xh).sum(0)
