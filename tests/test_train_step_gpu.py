"""The example's training step: every gradient of the block against the
float64 definitions of its parts put together, and a few steps that learn."""
import os
import sys

import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import training_oracle as T

from _common import TOL_BF16, rel_err

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _f(t):
    return t.double().cpu().numpy()


def test_gradients_of_the_block():
    import torch
    from train_step import Block
    b = Block(T=200, H=128, E=8, I=64, top_k=2, V=301, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    tokens = torch.randint(0, 301, (200,), generator=g, device="cuda")
    targets = torch.randint(0, 301, (200,), generator=g, device="cuda")
    targets[::7] = -100
    loss = float(b.forward(tokens, targets))
    b.backward(tokens, targets)
    torch.cuda.synchronize()
    assert b.moe.device_status() == 0 and b.xent.device_status() == 0
    w = {k: _f(v) for k, v in b.w.items()}
    tk, tg = tokens.cpu().numpy(), targets.cpu().numpy()
    # the forward, in 64 bits, with the stored (bf16) activations at each seam
    n1, n2, h1, h0 = _f(b.n1), _f(b.n2), _f(b.h1), _f(b.h0)
    assert rel_err(n1, T.layer_norm(h0, w["gamma1"], w["beta1"], 1e-5)[0]) <= TOL_BF16
    idx, gate = O.route((b.n1.float() @ b.w["Wr"]).cpu().numpy(), 2)
    assert rel_err(_f(b.y), O.forward(n1, w["W13"], w["W2"], idx, gate)) <= TOL_BF16
    assert rel_err(n2, T.layer_norm(h1, w["gamma2"], w["beta2"], 1e-5)[0]) <= TOL_BF16
    want, _, mean = T.cross_entropy(n2, w["Wout"], tg)
    assert abs(loss - mean) <= 1e-4 * mean
    # the backward
    on = T.counted(tg, 301, -100)
    dn2, dWout, _ = T.cross_entropy_backward(n2, w["Wout"], tg, np.full(200, 1.0 / on.sum()))
    dh1, dg2, db2 = T.layer_norm_backward(dn2, h1, w["gamma2"], 1e-5)
    m = O.backward(n1, w["W13"], w["W2"], idx, gate, dh1)
    dl = O.route_backward(gate, idx, m["dgate"], 8)
    dn1 = m["dX"] + dl @ w["Wr"].T
    dh0, dg1, db1 = T.layer_norm_backward(dn1, h0, w["gamma1"], 1e-5)
    dtable = np.zeros_like(w["table"])
    np.add.at(dtable, tk, dh0 + dh1)
    # each seam rounds to bf16: up to five of them between the loss and the table
    for k, ref in dict(Wout=dWout, gamma2=dg2, beta2=db2, W13=m["dW13"], W2=m["dW2"], Wr=n1.T @ dl, gamma1=dg1,
                       beta1=db1, table=dtable).items():
        assert rel_err(_f(b.g[k]), ref) <= TOL_BF16, k
    # clipping scales them all by the same factor
    norm = T.grad_norm([_f(v) for v in b.g.values()])
    before = {k: _f(v) for k, v in b.g.items()}
    b.clip.clip(0.5 * norm)
    torch.cuda.synchronize()
    assert abs(float(b.clip.norm) - norm) <= 1e-5 * norm
    for k, v in b.g.items():
        assert rel_err(_f(v), 0.5 * before[k]) <= 2.0 ** -8, k


def test_steps_learn():
    import torch
    from train_step import Block
    b = Block(T=512, H=128, E=8, I=64, top_k=2, V=97, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    table = torch.randperm(97, generator=g, device="cuda")
    losses, norms = [], []
    for _ in range(25):
        tokens = torch.randint(0, 97, (512,), generator=g, device="cuda")
        loss, norm = b.step(tokens, table[tokens], 1.0, 1.0)
        losses.append(float(loss))
        norms.append(float(norm))
    assert np.isfinite(losses).all() and np.isfinite(norms).all()
    assert losses[-1] < 0.5 * losses[0]
    assert b.moe.device_status() == b.xent.device_status() == b.clip.device_status() == 0
