"""Activations kept in 8 bits: what is restored, the backward pass from it, and
the operators around the layer put together.

X and h13 come back as the values of their codes, exactly.  act = silu(u) v (times
the gate) is computed with a fast exponential, relative error (4 + 2 |u|) U, and
a quotient and two products: within U (16 + 4 |u|), and one rounding when stored."""
import numpy as np
import pytest

from oracle import moe_oracle as M
from oracle import training_oracle as O

from _common import TOL_BF16, rel_err

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _f64(t):
    return t.double().cpu().numpy()


def _inputs(T, H, E, I, dtype, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)
    return dict(X=make(T, H), W13=make(E, H, 2 * I, scale=H ** -0.5), W2=make(E, I, H, scale=I ** -0.5), dY=make(T, H),
                logits=torch.randn((T, E), generator=g, device="cuda"))


def _codes(m):
    return M.dequantize_mxfp8(m.codes.cpu().numpy(), m.scales.cpu().numpy(), 1)


def _backward(X, h13, gate, idx, W13, W2, dY):
    """The layer's gradients at these X and h13 [T k, 2I], expert by expert."""
    T, k = idx.shape
    I = W2.shape[1]
    out = dict(dX=np.zeros(dY.shape), dW13=np.zeros(W13.shape), dW2=np.zeros(W2.shape), dgate=np.zeros((T, k)))
    u, v = h13[:, :I], h13[:, I:]
    sg = M.sigmoid(u)
    for e in range(len(W13)):
        a = np.nonzero(idx.reshape(-1) == e)[0]
        t, w = a // k, gate.reshape(-1)[a][:, None]
        A = u[a] * sg[a] * v[a]
        D = dY[t] @ W2[e].T
        out["dgate"].reshape(-1)[a] = (A * D).sum(1)
        dA = w * D
        dh = np.concatenate([dA * v[a] * sg[a] * (1 + u[a] * (1 - sg[a])), dA * u[a] * sg[a]], 1)
        out["dW2"][e] = (w * A).T @ dY[t]
        out["dW13"][e] = X[t].T @ dh
        np.add.at(out["dX"], t, dh @ W13[e].T)
    return out


# the last: rows of more than one unit of the kernels, and experts without a token
CASES = [("bf16", 1, 64, 4, 64, 4), ("f32", 100, 64, 8, 64, 2), ("bf16", 333, 320, 6, 192, 3), ("f32", 257, 192, 16, 128, 1),
         ("fp8_bwd", 200, 256, 8, 384, 2), ("bf16", 130, 2112, 40, 1088, 2)]


@pytest.mark.parametrize("mode,T,H,E,I,k", CASES)
def test_restored_activations_and_gradients(mode, T, H, E, I, k):
    import torch
    from mixture_experts_layer_18_gb300.layer import MoELayer
    L = MoELayer(T, H, E, I, k, mode=mode)
    d = _inputs(T, H, E, I, L.dtype)
    if E == 40:
        d["logits"][:, ::3] = -float("inf")
    io = L.empty_io()
    L.route(d["logits"])
    L.forward(d["X"], d["W13"], d["W2"], io["Y"])
    torch.cuda.synchronize()
    n = int(L.padded_offsets[-1])
    before = L.h13[:n].clone()
    act = L.act[:n].clone()
    ck = L.checkpoint()
    for t in (ck.x.codes, ck.x.scales, ck.h13.codes, ck.h13.scales):
        t.fill_(255)
    L.save(ck, d["X"])
    tail = 9.0
    L.x_perm.fill_(5.0)
    L.h13.fill_(5.0)
    L.act.fill_(5.0)
    L.x_perm[n:], L.h13[n:], L.act[n:] = tail, tail, tail
    L.restore(ck)
    torch.cuda.synchronize()
    assert L.device_status() == 0
    # codes: the rule on what the forward had
    row = L.row_of_assign.cpu().numpy()
    for m, src in ((ck.x, _f64(d["X"])), (ck.h13, _f64(before)[row])):
        codes, scales = M.quantize_mxfp8(src, 1)
        # (-0 has a code of its own)
        assert np.array_equal(_codes(m), M.dequantize_mxfp8(codes, scales, 1))
        assert np.array_equal(m.scales.cpu().numpy(), scales)
    X, h = _codes(ck.x), _codes(ck.h13)
    a = L.assign_of_row.cpu().numpy()[:n]
    real = a >= 0
    want = np.zeros((n, H))
    want[real] = X[a[real] // k]
    assert np.array_equal(_f64(L.x_perm[:n]), want)
    want = np.zeros((n, 2 * I))
    want[real] = h[a[real]]
    assert np.array_equal(_f64(L.h13[:n]), want)
    u, v = want[:, :I], want[:, I:]
    A = M.silu(u) * v
    if mode == "bf16":
        g = np.zeros(n)
        g[real] = _f64(L.gate).reshape(-1)[a[real]]
        A = A * g[:, None]
    st = U if mode == "f32" else 2.0 ** -8
    got = _f64(L.act[:n])
    assert (np.abs(got - A) <= np.abs(A) * (st + (1 + st) * U * (16 + 4 * np.abs(u))) + 1e-37).all()
    assert not got[~real].any()
    # the rows behind the last expert's stay as they were
    assert (L.x_perm[n:] == tail).all() and (L.h13[n:] == tail).all() and (L.act[n:] == tail).all()
    # what the codes are off: at most 2^-4 of a value, or half a step of the block's smallest, or
    # (values that saturate) an eighth
    assert (np.abs(_f64(L.h13[:n]) - _f64(before)) <= np.abs(_f64(before)) / 8 +
            np.abs(_f64(before)).reshape(n, -1, 32).max(2).repeat(32, 1) * 2.0 ** -17).all()
    L.backward(d["dY"], d["W13"], d["W2"], io["dX"], io["dW13"], io["dW2"], io["dgate"])
    torch.cuda.synchronize()
    assert L.device_status() == 0
    ref = _backward(X, h, _f64(L.gate), L.topk_idx.cpu().numpy(), _f64(d["W13"]), _f64(d["W2"]), _f64(d["dY"]))
    for name, r in ref.items():
        if mode == "fp8_bwd":
            # its products read codes too, of up to four tensors in a row (dY, W2, dh13, W13), each off by at most
            # 2^-4 of a value, uniformly (2^-4 / sqrt(3) of a norm): their sum bounds the gradient's
            assert np.linalg.norm(_f64(io[name]) - r) <= 4 * 2.0 ** -4 / 3 ** 0.5 * np.linalg.norm(r), name
        else:
            assert rel_err(_f64(io[name]), r) <= TOL_BF16, name


def test_layers_share_their_buffers():
    """Two layers with weights and routers of their own, one MoELayer: the second
    forward overwrites what the first saved; each backward has its own again."""
    import torch
    from mixture_experts_layer_18_gb300.layer import MoELayer
    from mixture_experts_layer_18_gb300.training import Router
    T, H, E, I, k = 300, 128, 8, 128, 2
    L = MoELayer(T, H, E, I, k)
    d = [_inputs(T, H, E, I, torch.bfloat16, s) for s in (1, 2)]
    routers = [Router(T, E, k, score="sigmoid", groups=4, top_groups=2, group_top=2, scale=1.5) for _ in d]
    cks = [L.checkpoint() for _ in d]

    def forward(i):
        io = L.empty_io()
        routers[i].forward(d[i]["logits"])
        L.forward(d[i]["X"], d[i]["W13"], d[i]["W2"], io["Y"], route=routers[i])
        L.save(cks[i], d[i]["X"], route=routers[i])
        return io

    def backward(i, io):
        L.restore(cks[i], route=routers[i])
        L.backward(d[i]["dY"], d[i]["W13"], d[i]["W2"], io["dX"], io["dW13"], io["dW2"], io["dgate"], route=routers[i])
        torch.cuda.synchronize()
        return {n: t.clone() for n, t in io.items()}
    alone = [backward(i, forward(i)) for i in (0, 1)]
    io = [forward(0), forward(1)]
    got = [backward(1, io[1]), backward(0, io[0])][::-1]
    assert L.device_status() == 0
    for i in (0, 1):
        for n in alone[i]:
            assert torch.equal(alone[i][n], got[i][n]), (i, n)
        idx, gate = O.route_by_scores(d[i]["logits"].cpu().numpy(), None, k, "sigmoid", 4, 2, 2, True, 1.5)
        assert np.array_equal(routers[i].topk_idx.cpu().numpy(), idx)
        Y = M.forward(_f64(d[i]["X"]), _f64(d[i]["W13"]), _f64(d[i]["W2"]), idx, gate)
        assert rel_err(_f64(got[i]["Y"]), Y) <= TOL_BF16


def test_a_block_of_all_of_them():
    """h = x + residual, its norm in bf16 for the layer and in 8 bits for the
    backward, sigmoid routing in groups, the experts, and back to x and the
    router's logits; then as one captured graph."""
    import torch
    from mixture_experts_layer_18_gb300.layer import MoELayer
    from mixture_experts_layer_18_gb300.training import RMSNorm, Router
    T, H, E, I, k = 260, 128, 16, 64, 3
    g = torch.Generator(device="cuda").manual_seed(5)
    d = _inputs(T, H, E, I, torch.bfloat16, 5)
    res, gamma = torch.randn((T, H), generator=g, device="cuda").bfloat16(), torch.rand(H, generator=g, device="cuda") + 0.5
    Wr = torch.randn((H, E), generator=g, device="cuda") / H ** 0.5
    bias = 0.01 * torch.randn(E, generator=g, device="cuda")
    norm, L = RMSNorm(T, H, weight_dtype=torch.float32), MoELayer(T, H, E, I, k)
    how = dict(score="sigmoid", groups=4, top_groups=2, group_top=2, scale=2.0)
    router, ck = Router(T, E, k, **how), L.checkpoint()
    n, io = norm.empty_io(), L.empty_io()
    dl, logits, new_bias = (torch.empty(s, device="cuda") for s in ((T, E), (T, E), (E,)))
    dn = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")

    def step():
        norm.forward(d["X"], gamma, n["y"], residual=res, h=n["h"], encoded=ck.x)
        torch.mm(n["y"].float(), Wr, out=logits)
        router.forward(logits, bias)
        L.forward(n["y"], d["W13"], d["W2"], io["Y"], route=router)
        L.save(ck, route=router)
        L.saved.zero_()                                         # another layer's turn
        L.restore(ck, route=router)
        L.backward(d["dY"], d["W13"], d["W2"], io["dX"], io["dW13"], io["dW2"], io["dgate"], route=router)
        router.backward(logits, io["dgate"], dl)
        torch.add(io["dX"], (dl @ Wr.T).bfloat16(), out=dn)
        norm.backward(dn, n["h"], gamma, n["dx"], n["dgamma"], dh=d["dY"])
        router.update_bias(bias, 1e-3, out=new_bias)
    step()
    torch.cuda.synchronize()
    assert L.device_status() == router.device_status() == 0
    # each part at the stored values that it read
    h, y, rstd = O.rms_norm(_f64(d["X"]), _f64(res), _f64(gamma), 1e-6)
    assert rel_err(_f64(n["y"]), y) <= TOL_BF16 and rel_err(_f64(n["h"]), h) <= TOL_BF16
    lg = logits.cpu().numpy()
    idx, gate = O.route_by_scores(lg, bias.cpu().numpy(), k, **how)
    assert np.array_equal(router.topk_idx.cpu().numpy(), idx)
    assert rel_err(_f64(io["Y"]), M.forward(_f64(n["y"]), _f64(d["W13"]), _f64(d["W2"]), idx, gate)) <= TOL_BF16
    b = _backward(_codes(ck.x), _codes(ck.h13), gate, idx, _f64(d["W13"]), _f64(d["W2"]), _f64(d["dY"]))
    for name in ("dX", "dW13", "dW2", "dgate"):
        assert rel_err(_f64(io[name]), b[name]) <= TOL_BF16, name
    want = O.route_by_scores_backward(lg, idx, gate, _f64(io["dgate"]), "sigmoid", True, 2.0)
    assert rel_err(_f64(dl), want) <= 1e-4
    dx, dg = O.rms_norm_backward(_f64(dn), _f64(n["h"]), _f64(gamma), rstd, _f64(d["dY"]))
    assert rel_err(_f64(n["dx"]), dx) <= TOL_BF16 and rel_err(_f64(n["dgamma"]), dg) <= TOL_BF16
    assert np.allclose(_f64(new_bias), O.balance_bias(router.counts.cpu().numpy(), 1e-3, _f64(bias)), atol=1e-8)
    # 8 bits against none: the same backward from what the forward saved itself
    exact = M.backward(_f64(n["y"]), _f64(d["W13"]), _f64(d["W2"]), idx, gate, _f64(d["dY"]))
    for name in ("dX", "dW13", "dW2", "dgate"):
        # both factors of a product carry codes off by at most 2^-4, uniformly: 2^-4 / sqrt(3) of a norm, and the
        # activation's derivative up to twice that
        off = np.linalg.norm(_f64(io[name]) - exact[name]) / np.linalg.norm(exact[name])
        assert off <= 4 * 2.0 ** -4 / 3 ** 0.5, name
    kept = [t.clone() for t in (io["Y"], io["dX"], io["dW13"], dl, n["dx"], n["dgamma"], new_bias)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(kept, (io["Y"], io["dX"], io["dW13"], dl, n["dx"], n["dgamma"], new_bias)):
        assert torch.equal(a, b)


def test_bad_rows_are_reported():
    """Row numbers outside the buffer are reported and skipped."""
    import torch
    from mixture_experts_layer_18_gb300 import MOE_ERR_BAD_INDEX
    from mixture_experts_layer_18_gb300.layer import MoELayer
    L = MoELayer(20, 64, 4, 64, 2)
    d = _inputs(20, 64, 4, 64, torch.bfloat16)
    io = L.empty_io()
    L.route(d["logits"])
    L.forward(d["X"], d["W13"], d["W2"], io["Y"])
    ck = L.checkpoint()
    keep = int(L.row_of_assign[5]), int(L.row_of_assign[9])
    for call in (lambda: L.save(ck, d["X"]), lambda: L.restore(ck)):
        L.row_of_assign[5], L.row_of_assign[9] = -4, 1 << 30
        L.clear_status()
        call()
        assert L.device_status() == MOE_ERR_BAD_INDEX
        L.row_of_assign[5], L.row_of_assign[9] = keep
        L.clear_status()
        call()
        assert L.device_status() == 0


def test_activations_past_32_bits():
    """More than 2^31 elements of h13: the last tokens' rows are their own."""
    import torch
    from mixture_experts_layer_18_gb300.layer import MoELayer
    T, H, E, I, k = 300_000, 64, 4, 2048, 2
    L = MoELayer(T, H, E, I, k, backward=False)
    g = torch.Generator(device="cuda").manual_seed(2)
    L.route(torch.randn((T, E), generator=g, device="cuda"))
    n = int(L.padded_offsets[-1])
    rows = L.row_of_assign[-40:].long()
    L.h13.zero_()
    part = torch.randn((40, 2 * I), generator=g, device="cuda").bfloat16()
    L.h13[rows] = part
    X = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    ck = L.checkpoint()
    L.save(ck, X)
    L.h13.fill_(3.0)
    L.act.fill_(3.0)
    L.restore(ck)
    torch.cuda.synchronize()
    assert L.device_status() == 0
    want = M.dequantize_mxfp8(*M.quantize_mxfp8(_f64(part), 1), 1)
    assert np.array_equal(_f64(L.h13[rows]), want)
    assert not L.h13[:n].index_fill(0, rows, 0).any() and not L.act[:n].index_fill(0, rows, 0).any()
    x = M.dequantize_mxfp8(*M.quantize_mxfp8(_f64(X[-20:]), 1), 1)
    assert np.array_equal(_f64(L.x_perm[rows]), x.repeat(k, 0))
