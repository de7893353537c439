"""Host-side checks of routing by scores, the RMS norm, MXFP8 rows and the
checkpoints: what is refused before any launch (CPU: the pointers are fake and
never used), and the Python side on host tensors."""
import math
import threading

import pytest
import torch

import mixture_experts_layer_18_gb300 as M
from mixture_experts_layer_18_gb300 import layer, training

P = 1 << 20          # a fake device address, aligned for every type
BAD = M.MOE_ERR_INVALID_ARG


def _router(**kw):
    base = dict(T=4, E=32, top_k=4, ld=32, type=M.MOE_TYPE_F32, score=M.MOE_SCORE_SIGMOID, groups=4, top_groups=2,
                group_top=2, renormalise=1, scale=1.0)
    base.update(kw)
    return M.moe_router_dims(*base.values())


def _route(**kw):
    return M.moe_route_out(*{**dict(i=P, g=P, c=P, o=P, p=P, r=P, a=P), **kw}.values())


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(E=0), dict(E=1025, ld=1025), dict(top_k=0), dict(top_k=33, E=64, ld=64, groups=1, top_groups=1),
    dict(ld=31), dict(type=2), dict(score=2), dict(score=-1), dict(groups=0), dict(groups=5), dict(groups=64, E=64, ld=64),
    dict(top_groups=0), dict(top_groups=5), dict(group_top=0), dict(group_top=3), dict(groups=32, group_top=2),
    dict(top_k=17), dict(scale=0.0), dict(scale=2.0 ** -65), dict(scale=2.0 ** 65), dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan),
    dict(T=1 << 29, top_k=4)])
def test_router_dims_refused(bad):
    d = _router(**bad)
    assert M.moe_router_workspace_size(d) == 0
    assert M.moe_router(d, P, P, _route(), P, 1 << 40, P, None) == BAD
    assert M.moe_router_backward(d, _route(), P, P, P, P, None) == BAD


def test_router_pointers_refused():
    d = _router()
    need = M.moe_router_workspace_size(d)
    assert need > 0
    ok = dict(l=P, b=P, o=_route(), ws=P, n=need, st=P)
    for bad in (dict(l=None), dict(l=P + 2), dict(b=P + 2), dict(ws=None), dict(ws=P + 8), dict(n=need - 1),
                dict(st=None), dict(st=P + 4), *[dict(o=_route(**{k: v})) for k in "igcopra" for v in (None, P + 4)]):
        assert M.moe_router(d, *{**ok, **bad}.values(), None) == BAD, bad
    ok = dict(o=_route(), l=P, dg=P, dl=P, st=P)
    for bad in (dict(o=_route(i=None)), dict(o=_route(g=P + 4)), dict(l=None), dict(dg=None), dict(dg=P + 2),
                dict(dl=None), dict(dl=P + 1), dict(st=None)):
        assert M.moe_router_backward(d, *{**ok, **bad}.values(), None) == BAD, bad
    assert M.moe_router_backward(_router(T=0), _route(), None, None, None, P, None) == M.MOE_OK
    ok = dict(E=8, c=P, rate=0.1, b=P, o=P)
    for bad in (dict(E=0), dict(E=1025), dict(c=None), dict(rate=math.inf), dict(rate=math.nan), dict(b=None), dict(o=None),
                dict(o=P + 2)):
        assert M.moe_balance_bias(*{**ok, **bad}.values(), None) == BAD, bad


def _rms(**kw):
    base = dict(T=4, H=64, ld_x=64, ld_residual=64, ld_h=64, ld_y=64, ld_dh=64, ld_dx=64, x_type=M.MOE_TYPE_BF16,
                w_type=M.MOE_TYPE_F32, eps=1e-6)
    base.update(kw)
    return M.moe_rms_dims(*base.values())


@pytest.mark.parametrize("bad", [dict(T=-1), dict(H=0), dict(ld_x=63), dict(ld_residual=0), dict(ld_h=63), dict(ld_y=63),
                                 dict(ld_dh=63), dict(ld_dx=63), dict(x_type=2), dict(w_type=-1), dict(eps=-1.0),
                                 dict(eps=math.inf), dict(eps=math.nan)])
def test_rms_dims_refused(bad):
    d = _rms(**bad)
    assert M.moe_rms_norm_workspace_size(d) == 0
    assert M.moe_rms_norm(d, P, P, P, P, 2 * P, P, P, P, None) == BAD
    assert M.moe_rms_norm_backward(d, P, P, P, P, P, P, P, P, 1 << 30, None) == BAD


def test_rms_pointers_refused():
    d = _rms()
    ok = dict(x=P, r=P, g=P, h=P, y=2 * P, q=P, s=P, rstd=P)
    for bad in (dict(x=None), dict(x=P + 1), dict(r=P + 1), dict(g=P + 2), dict(h=P + 1), dict(y=P + 1), dict(h=2 * P),
                dict(r=None), dict(q=P + 8), dict(q=None), dict(s=None), dict(rstd=P + 2)):
        assert M.moe_rms_norm(d, *{**ok, **bad}.values(), None) == BAD, bad
    assert M.moe_rms_norm(_rms(H=48), *ok.values(), None) == BAD               # codes need blocks of 32
    assert M.moe_rms_norm(_rms(T=0), *[None] * 8, None) == M.MOE_OK
    need = M.moe_rms_norm_workspace_size(d)
    ok = dict(dy=P, h=P, dh=P, g=P, rstd=P, dx=P, dg=P, ws=P, n=need)
    for bad in (dict(dy=None), dict(h=None), dict(dh=P + 1), dict(g=P + 2), dict(rstd=None), dict(dx=None), dict(dx=P + 1),
                dict(dg=P + 2), dict(ws=None), dict(ws=P + 8), dict(n=need - 1)):
        assert M.moe_rms_norm_backward(d, *{**ok, **bad}.values(), None) == BAD, bad


def test_dequantize_refused():
    ok = dict(q=P, s=P, R=4, C=64, ld=64, type=M.MOE_TYPE_BF16, dst=P)
    for bad in (dict(q=None), dict(q=P + 8), dict(s=None), dict(R=-1), dict(C=48), dict(C=-32), dict(ld=63), dict(type=2),
                dict(dst=None), dict(dst=P + 1)):
        assert M.moe_dequantize_mxfp8(*{**ok, **bad}.values(), None) == BAD, bad
    assert M.moe_dequantize_mxfp8(None, None, 0, 64, 64, M.MOE_TYPE_F32, None, None) == M.MOE_OK


def test_checkpoints_refused():
    def dims(**kw):
        return M.moe_dims(*{**dict(T=4, H=64, E=4, I=64, k=2, mode=M.MOE_BF16, save=1), **kw}.values())
    need = M.moe_saved_layout_of(dims()).total

    def both(d, X=P, r=None, saved=P, n=need, c=None, st=P):
        r, c = r or _route(), c or M.moe_checkpoint(P, P, P, P)
        return {M.moe_checkpoint_save(d, X, r, saved, n, c, st, None), M.moe_checkpoint_restore(d, c, r, saved, n, st, None)}
    for bad in (dict(T=-1), dict(H=65), dict(k=5), dict(save=0), dict(mode=9)):
        assert both(dims(**bad), n=1 << 40) == {BAD}, bad
    assert both(dims(mode=M.MOE_MXFP8, H=128, I=384), n=1 << 40) == {M.MOE_ERR_UNSUPPORTED}
    for bad in (dict(saved=None), dict(saved=P + 8), dict(n=need - 1), dict(st=None), dict(r=_route(r=None)),
                dict(r=_route(p=None)), *[dict(c=M.moe_checkpoint(*[None if i == j else P for j in range(4)])) for i in range(4)]):
        assert both(dims(), **bad) == {BAD}, bad
    assert M.moe_checkpoint_save(dims(), P + 8, _route(), P, need, M.moe_checkpoint(P, P, P, P), P, None) == BAD


# ------------------------------------------------------------ the Python side
@pytest.fixture
def host(monkeypatch):
    """Ops on host memory; returns the module."""
    def device(self, _):
        self.index, self.device = -1, torch.device("cpu")
    monkeypatch.setattr(training._Op, "_device", device)
    monkeypatch.setattr(training._Op, "_current", lambda self, stream: 0)
    return training


def test_sizes_are_checked(host):
    big = 1 << 32
    for make in (lambda: host.Router(big + 4, 8, 2), lambda: host.Router(4, big + 8, 2), lambda: host.Router(4, 8, big + 2),
                 lambda: host.Router(4, 8, 2, groups=big + 1), lambda: host.RMSNorm(big + 4, 64), lambda: host.RMSNorm(4, big),
                 lambda: host.MXRows(big, 32), lambda: host.MXRows(4, 48), lambda: host.Router(4, 8, 2, score="linear"),
                 lambda: host.Router(4, 8, 2, dtype=torch.float16), lambda: host.RMSNorm(4, 64, dtype=torch.float16),
                 lambda: host.Router(4, 8, 9), lambda: host.Router(4, 8, 2, scale=0.0), lambda: host.Router(4, 8, 2, groups=3)):
        with pytest.raises(M.MoEError):
            make()


def test_tensors_are_checked(host, monkeypatch):
    for name in ("moe_router", "moe_router_backward", "moe_balance_bias", "moe_rms_norm", "moe_rms_norm_backward",
                 "moe_quantize_mxfp8", "moe_dequantize_mxfp8"):
        monkeypatch.setattr(host, name, lambda *a: 0)
    r = host.Router(4, 8, 2)
    l, b, dg, dl = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4, 2), torch.zeros(4, 8)
    r.forward(torch.zeros(4, 11)[:, :8], b)
    r.backward(l, dg, dl)
    r.update_bias(b, 0.1)
    n, m = host.RMSNorm(4, 64), host.MXRows(4, 64)
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    n.forward(x, w, x, residual=x, h=x.clone(), encoded=m)
    n.forward(x, None, encoded=m)
    n.backward(x, x, w, x, w, dh=x)
    m.decode(x)
    m.decode(x.float())
    for call in (lambda: r.forward(l.double()), lambda: r.forward(l[:3]), lambda: r.forward(l.T.contiguous().T),
                 lambda: r.forward(l, b.double()), lambda: r.forward(l, b[:7]), lambda: r.backward(l, dg[:, :1], dl),
                 lambda: r.backward(l, dg, torch.zeros(4, 9)[:, :8]), lambda: r.update_bias(b[:4], 0.1),
                 lambda: r.update_bias(b, 0.1, out=b.double()), lambda: r.forward(None),
                 lambda: n.forward(x, w, x, h=x), lambda: n.forward(x.float(), w, x), lambda: n.forward(x, w.float(), x),
                 lambda: n.forward(x, w, x, residual=x[:3]), lambda: n.forward(x, w, x, encoded=host.MXRows(4, 32)),
                 lambda: n.forward(x, w, x, encoded=host.MXRows(3, 64)), lambda: n.backward(x, x, w, x, w.float()),
                 lambda: n.backward(x, x, w, x, dh=x.float()), lambda: m.decode(x.half()), lambda: m.decode(x[:2]),
                 lambda: m.encode(x.float()), lambda: host.RMSNorm(4, 64, backward=False).backward(x, x, w, x)):
        with pytest.raises(M.MoEError):
            call()


def test_calls_of_two_threads_keep_their_strides(host, monkeypatch):
    meet, seen = threading.Barrier(2, timeout=10), {}

    def library(d, x, *a):
        meet.wait()                     # (both callers have described their rows)
        seen[x] = d.ld if hasattr(d, "ld") else (d.ld_x, d.ld_y)
        return 0
    monkeypatch.setattr(host, "moe_router", library)
    monkeypatch.setattr(host, "moe_rms_norm", library)
    r, n = host.Router(6, 64, 2), host.RMSNorm(6, 64, dtype=torch.float32)
    x = [torch.zeros((6, 64 + p))[:, :64] for p in (8, 24, 8, 24)]
    for calls in ([lambda i=i: r.forward(x[i]) for i in (0, 1)], [lambda i=i: n.forward(x[i], None, x[i]) for i in (2, 3)]):
        threads = [threading.Thread(target=c) for c in calls]
        for t in threads:
            t.start()
        for t in threads:
            t.join(20)
    assert [seen[t.data_ptr()] for t in x] == [72, 88, (72, 72), (88, 88)]


def test_memory_whose_address_is_recorded_stays(host):
    import weakref
    for op, names in ((host.Router(4, 8, 2), ("topk_idx", "gate", "counts", "offsets", "padded_offsets", "row_of_assign",
                                              "assign_of_row", "ws", "status")),
                      (host.RMSNorm(4, 64), ("rstd", "ws")), (host.MXRows(4, 64), ("codes", "scales", "status"))):
        held = {k: weakref.ref(getattr(op, k)) for k in names}
        for k in names:
            setattr(op, k, None)
        assert all(r() is not None for r in held.values()), op


def test_layer_calls_are_checked(host, monkeypatch):
    seen = []
    for name in ("moe_forward", "moe_backward", "moe_checkpoint_save", "moe_checkpoint_restore"):
        monkeypatch.setattr(layer, name, lambda *a, name=name: seen.append((name, a)) or 0)
    monkeypatch.setattr(layer, "_stream", lambda s: 0)
    monkeypatch.setattr(layer, "_current_device", lambda: None)
    L = layer.MoELayer(4, 64, 4, 64, 2, device="cpu")
    r, ck = host.Router(4, 4, 2), L.checkpoint()
    X = torch.zeros((4, 64), dtype=torch.bfloat16)
    L.save(ck, X, route=r)
    L.save(ck)
    L.restore(ck, route=r)
    L.forward(X, X, X, X, route=r)
    L.backward(X, X, X, X, X, X, X, route=r)
    assert seen[0][1][2] is r.route_out and seen[1][1][1] is None and seen[1][1][2] is L.route_out
    assert seen[2][1][2] is r.route_out and seen[3][1][4] is r.route_out and seen[4][1][4] is r.route_out
    other = layer.MoELayer(4, 128, 4, 64, 2, device="cpu")
    for call in (lambda: L.save(ck, X.float()), lambda: L.save(ck, X[:3]), lambda: L.save(other.checkpoint(), X),
                 lambda: L.restore(other.checkpoint()), lambda: L.save(ck, X, route=host.Router(4, 8, 2)),
                 lambda: L.forward(X, X, X, X, route=host.Router(5, 4, 2)),
                 lambda: layer.MoELayer(4, 128, 4, 384, 2, mode="mxfp8", device="cpu").checkpoint()):
        with pytest.raises(M.MoEError):
            call()
    monkeypatch.setattr(layer, "_current_device", lambda: 3)
    with pytest.raises(M.MoEError):
        L.restore(ck)
