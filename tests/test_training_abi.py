"""Host-side checks of the training-step operators: what is refused before
any launch (CPU: the pointers are fake and never used)."""
import ctypes
import math

import pytest

import mixture_experts_layer_18_gb300 as M

P = 1 << 20          # a fake device address, aligned for every type


def _norm(**kw):
    base = dict(T=4, H=64, ld_x=64, ld_y=64, ld_dx=64, x_type=M.MOE_TYPE_BF16, w_type=M.MOE_TYPE_F32, eps=1e-5)
    base.update(kw)
    return M.moe_norm_dims(*base.values())


@pytest.mark.parametrize("bad", [dict(T=-1), dict(H=0), dict(ld_x=63), dict(ld_y=0), dict(ld_dx=63),
                                 dict(x_type=2), dict(w_type=-1), dict(eps=-1.0), dict(eps=math.inf),
                                 dict(eps=math.nan)])
def test_norm_dims_refused(bad):
    d = _norm(**bad)
    assert M.moe_layer_norm_workspace_size(d) == 0
    assert M.moe_layer_norm(d, P, P, P, P, P, P, None) == M.MOE_ERR_INVALID_ARG
    assert M.moe_layer_norm_backward(d, P, P, P, P, P, P, P, P, P, 1 << 30, None) == M.MOE_ERR_INVALID_ARG


def test_norm_pointers_refused():
    d = _norm()
    ok = dict(x=P, g=P, b=P, y=P, m=P, r=P)
    for bad in (dict(x=None), dict(y=None), dict(x=P + 1), dict(y=P + 1), dict(g=P + 2), dict(b=P + 1), dict(m=P + 2),
                dict(r=P + 1)):
        a = {**ok, **bad}
        assert M.moe_layer_norm(d, a["x"], a["g"], a["b"], a["y"], a["m"], a["r"], None) == M.MOE_ERR_INVALID_ARG, bad
    need = M.moe_layer_norm_workspace_size(d)
    ok = dict(dy=P, x=P, g=P, m=P, r=P, dx=P, dg=P, db=P, ws=P, n=need)
    for bad in (dict(dy=None), dict(x=None), dict(m=None), dict(r=None), dict(dx=None), dict(dx=P + 1), dict(dg=P + 2),
                dict(db=P + 1), dict(ws=None), dict(ws=P + 8), dict(n=need - 1)):
        a = {**ok, **bad}
        rc = M.moe_layer_norm_backward(d, a["dy"], a["x"], a["g"], a["m"], a["r"], a["dx"], a["dg"], a["db"], a["ws"],
                                       a["n"], None)
        assert rc == M.MOE_ERR_INVALID_ARG, bad
    assert M.moe_layer_norm(_norm(T=0), None, None, None, None, None, None, None) == M.MOE_OK   # nothing to do


def _xent(**kw):
    base = dict(T=4, H=64, V=100, ld_x=64, ld_w=64, ignore_index=-100, index_type=M.MOE_INDEX_I64)
    base.update(kw)
    return M.moe_xent_dims(*base.values())


@pytest.mark.parametrize("bad,code", [
    (dict(T=-1), M.MOE_ERR_INVALID_ARG), (dict(V=0), M.MOE_ERR_INVALID_ARG), (dict(H=0), M.MOE_ERR_INVALID_ARG),
    (dict(ld_x=56), M.MOE_ERR_INVALID_ARG), (dict(ld_w=56), M.MOE_ERR_INVALID_ARG),
    (dict(index_type=2), M.MOE_ERR_INVALID_ARG), (dict(H=63), M.MOE_ERR_UNSUPPORTED),
    (dict(ld_x=68), M.MOE_ERR_UNSUPPORTED), (dict(ld_w=65), M.MOE_ERR_UNSUPPORTED),
    (dict(T=1 << 30, V=1 << 30), M.MOE_ERR_UNSUPPORTED)])
def test_xent_dims_refused(bad, code):
    d = _xent(**bad)
    assert M.moe_cross_entropy_workspace_size(d, M.MOE_WS_FORWARD) == 0
    assert M.moe_cross_entropy_workspace_size(d, M.MOE_WS_BACKWARD) == 0
    assert M.moe_cross_entropy(d, P, P, P, P, P, P, P, 1 << 40, P, None) == code
    assert M.moe_cross_entropy_backward(d, P, P, P, P, P, P, M.MOE_REDUCE_MEAN, P, P, P, 1 << 40, P, None) == code


def test_xent_pointers_refused():
    d = _xent()
    f, b = (M.moe_cross_entropy_workspace_size(d, w) for w in (M.MOE_WS_FORWARD, M.MOE_WS_BACKWARD))
    assert f > 0 and b > 0 and M.moe_cross_entropy_workspace_size(d, M.MOE_WS_ROUTE) == 0
    ok = dict(X=P, W=P, t=P, loss=P, lse=P, total=P, ws=P, n=f, st=P)
    for bad in (dict(X=None), dict(X=P + 8), dict(W=None), dict(W=P + 2), dict(t=None), dict(t=P + 4),
                dict(loss=None), dict(lse=P + 2), dict(total=None), dict(ws=None), dict(ws=P + 8), dict(n=f - 1),
                dict(st=None), dict(st=P + 4)):
        assert M.moe_cross_entropy(d, *{**ok, **bad}.values(), None) == M.MOE_ERR_INVALID_ARG, bad
    ok = dict(X=P, W=P, t=P, lse=P, total=P, dl=P, red=M.MOE_REDUCE_MEAN, dX=P, dW=P, ws=P, n=b, st=P)
    for bad in (dict(X=None), dict(W=P + 8), dict(t=P + 1), dict(lse=None), dict(total=None), dict(dl=None),
                dict(red=3), dict(red=-1), dict(dX=P + 8), dict(dW=P + 2), dict(ws=None), dict(n=b - 1), dict(st=None)):
        assert M.moe_cross_entropy_backward(d, *{**ok, **bad}.values(), None) == M.MOE_ERR_INVALID_ARG, bad


def _grads(*entries):
    return (M.moe_grad_tensor * len(entries))(*[M.moe_grad_tensor(*e) for e in entries])


def test_grads_refused():
    need = M.moe_grad_workspace_size(1)
    assert need > 0 and M.moe_grad_workspace_size(-1) == 0
    assert M.moe_grad_workspace_size(2000) > M.moe_grad_workspace_size(1)
    good = _grads((P, P, 8, M.MOE_TYPE_F32))
    for bad in (_grads((None, P, 8, M.MOE_TYPE_F32)), _grads((P + 2, P, 8, M.MOE_TYPE_F32)),
                _grads((P + 1, P, 8, M.MOE_TYPE_BF16)), _grads((P, P, -1, M.MOE_TYPE_F32)),
                _grads((P, P, 8, 2)), _grads((P, P, 1 << 47, M.MOE_TYPE_F32))):
        assert M.moe_grad_norm(bad, 1, P, P, need, P, None) == M.MOE_ERR_INVALID_ARG
        assert M.moe_clip_grads(bad, 1, 1.0, P, P, need, P, None) == M.MOE_ERR_INVALID_ARG
    for dst in (None, P + 2):                     # dst matters to clipping alone
        assert M.moe_clip_grads(_grads((P, dst, 8, M.MOE_TYPE_F32)), 1, 1.0, P, P, need, P, None) == \
            M.MOE_ERR_INVALID_ARG
    for limit in (-1.0, math.inf, math.nan):
        assert M.moe_clip_grads(good, 1, limit, P, P, need, P, None) == M.MOE_ERR_INVALID_ARG
    null = ctypes.POINTER(M.moe_grad_tensor)()
    assert M.moe_grad_norm(null, 1, P, P, need, P, None) == M.MOE_ERR_INVALID_ARG
    for a in (dict(count=-1), dict(norm=None), dict(norm=P + 2), dict(ws=None), dict(ws=P + 8), dict(n=need - 1),
              dict(st=None), dict(st=P + 8)):
        k = {**dict(count=1, norm=P, ws=P, n=need, st=P), **a}
        assert M.moe_grad_norm(good, k["count"], k["norm"], k["ws"], k["n"], k["st"], None) == \
            M.MOE_ERR_INVALID_ARG, a
