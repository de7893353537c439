"""Layer norm on the GPU against its float64 definition.

Tolerances.  U = 2^-24 is the unit roundoff of fp32; a stored type adds its
own (2^-8 for bf16, which has 8 significant bits).  A row's mean is a tree of
at most 64 additions deep, so its error is below 64 U max|x|, which moves a
normalised value by that times rstd; the same count covers the variance.  The
bounds below are those errors carried through the formulas, plus one rounding
to the stored type."""
import numpy as np
import pytest

from oracle import training_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


def _stored(dtype):
    import torch
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def _run(x, gamma, beta, dy, eps=EPS, params=True):
    """Forward and backward through the public class; float64 results."""
    import torch
    from mixture_experts_layer_18_gb300.training import LayerNorm
    T, H = x.shape
    wt = gamma.dtype if gamma is not None else x.dtype
    n = LayerNorm(T, H, dtype=x.dtype, weight_dtype=wt, eps=eps)
    io = n.empty_io()
    for t in io.values():
        t.fill_(7.0)
    n.forward(x, gamma, beta, io["y"])
    n.backward(dy, x, gamma, io["dx"], io["dgamma"] if params else None, io["dbeta"] if params else None)
    torch.cuda.synchronize()
    out = {k: v.double().cpu().numpy() for k, v in io.items()}
    out["mean"], out["rstd"] = n.mean.double().cpu().numpy(), n.rstd.double().cpu().numpy()
    return out


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _check(x, gamma, beta, dy, out, eps=EPS):
    X, G, B, D = _f64(x), _f64(gamma), _f64(beta), _f64(dy)
    g1 = 1.0 if G is None else G
    b1 = 0.0 if B is None else B
    y, mean, rstd = O.layer_norm(X, G, B, eps)
    dx, dg, db = O.layer_norm_backward(D, X, G, eps)
    h = O.layer_norm(X, None, None, eps)[0]
    big = np.abs(X).max(1)
    e = 64 * U * (1 + big * rstd + np.abs(h).max(1))     # error of a row's normalised values
    ux = _stored(x.dtype)
    assert (np.abs(out["mean"] - mean) <= 64 * U * big + 1e-30).all()
    assert (np.abs(out["rstd"] - rstd) <= 2 * e * rstd).all()
    tol = ux * np.abs(y) + (1 + ux) * (e[:, None] * (np.abs(g1) * (1 + np.abs(h))) + 4 * U * np.abs(b1))
    assert (np.abs(out["y"] - y) <= tol).all(), np.abs(out["y"] - y).max()
    g = np.abs(D * g1)
    m = g.mean(1)[:, None] + g
    m = m + (g * np.abs(h)).mean(1)[:, None] * (1 + np.abs(h)) * 2
    tol = ux * np.abs(dx) + (1 + ux) * 2 * e[:, None] * rstd[:, None] * m
    assert (np.abs(out["dx"] - dx) <= tol).all(), np.abs(out["dx"] - dx).max()
    uw = _stored(x.dtype if gamma is None else gamma.dtype)
    n = (64 + X.shape[0] / 128) * U                      # depth of a column's sum
    tol = uw * np.abs(dg) + (1 + uw) * (n + e.max()) * (np.abs(D) * (1 + np.abs(h))).sum(0)
    assert (np.abs(out["dgamma"] - dg) <= tol).all(), np.abs(out["dgamma"] - dg).max()
    tol = uw * np.abs(db) + (1 + uw) * n * np.abs(D).sum(0)
    assert (np.abs(out["dbeta"] - db) <= tol).all(), np.abs(out["dbeta"] - db).max()


def _make(T, H, dtype, wdtype, pad=0, off=0, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed + T * 1000 + H)

    def rows():
        buf = torch.full((T, H + pad + off), 1e4, dtype=dtype, device="cuda")
        v = buf[:, off:off + H]
        v.copy_(torch.randn((T, H), generator=g, device="cuda") * 1.5 + 0.25)
        return v
    x, dy = rows(), rows()
    w = (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wdtype)
    b = torch.randn(H, generator=g, device="cuda").to(wdtype)
    return x, w, b, dy


# one lane, part of a warp, whole warps, several rows a block, every width class of the
# fused kernels and the long rows past them; odd widths take the element-wise form
SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (33, 64), (129, 96), (1000, 256), (257, 264), (700, 513), (311, 1000),
          (400, 2049), (640, 4096), (97, 4104), (70, 5001), (65, 8192), (40, 8200), (33, 16384), (9, 16392), (5, 20001),
          (3, 40000), (200, 9001), (31, 12004), (17, 16377)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16/f32"])
def test_layer_norm_matches_definition(T, H, kind):
    import torch
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    wt = torch.bfloat16 if kind == "bf16" else torch.float32
    x, w, b, dy = _make(T, H, dt, wt)
    _check(x, w, b, dy, _run(x, w, b, dy))


@pytest.mark.parametrize("pad,off", [(8, 0), (24, 8), (7, 0), (5, 3)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_strided_rows(pad, off, dtype):
    import torch
    dt = getattr(torch, dtype)
    x, w, b, dy = _make(130, 520, dt, dt, pad, off)
    _check(x, w, b, dy, _run(x, w, b, dy))


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_tensors_at_different_offsets(dtype):
    """x, y, dy and dx that start at different places in their 16-byte vectors."""
    import torch
    from mixture_experts_layer_18_gb300.training import LayerNorm
    dt = getattr(torch, dtype)
    x, w, b, dy = _make(77, 300, dt, torch.float32, pad=3)
    flat = torch.zeros(77 * 300 + 5, dtype=dt, device="cuda")
    n = LayerNorm(77, 300, dtype=dt, weight_dtype=torch.float32)
    y, dx = flat[1:1 + 77 * 300].view(77, 300), torch.zeros((77, 301), dtype=dt, device="cuda")[:, 1:]
    dg, db = torch.zeros_like(w), torch.zeros_like(w)
    n.forward(x, w, b, y)
    n.backward(dy, x, w, dx, dg, db)
    torch.cuda.synchronize()
    out = dict(y=_f64(y), dx=_f64(dx), dgamma=_f64(dg), dbeta=_f64(db), mean=_f64(n.mean), rstd=_f64(n.rstd))
    _check(x, w, b, dy, out)
    assert flat[0] == 0 and not flat[1 + 77 * 300:].any()


def test_many_rows():
    import torch
    x, w, b, dy = _make(20011, 192, torch.float32, torch.bfloat16)
    _check(x, w, b, dy, _run(x, w, b, dy))


def test_without_weights():
    import torch
    x, w, b, dy = _make(50, 320, torch.bfloat16, torch.float32)
    _check(x, None, None, dy, _run(x, None, None, dy))
    out = _run(x, w, b, dy, params=False)                # dgamma and dbeta left out, untouched
    assert (out["dgamma"] == 7).all() and (out["dbeta"] == 7).all()
    ref = O.layer_norm_backward(_f64(dy), _f64(x), _f64(w), EPS)[0]
    assert np.abs(out["dx"] - ref).max() <= 2.0 ** -8 * np.abs(ref).max()


def test_mean_much_larger_than_the_spread():
    """The variance comes from centred values: a common offset of 1000 spreads
    costs what the rounding of the mean costs, not its square."""
    import torch
    x, w, b, dy = _make(64, 1024, torch.float32, torch.float32)
    x = x + 1500.0
    _check(x, w, b, dy, _run(x, w, b, dy))


def test_constant_rows_and_zeros():
    import torch
    x, w, b, dy = _make(6, 128, torch.float32, torch.float32)
    x[0] = 0.0
    x[1] = 5.0
    out = _run(x, w, b, dy)
    _check(x, w, b, dy, out)
    assert np.array_equal(out["y"][0], _f64(b)) and np.array_equal(out["y"][1], _f64(b))


def test_variance_past_fp32():
    """A row whose variance overflows fp32 has rstd 0, as the formula says: y is beta."""
    import torch
    x, w, b, dy = _make(5, 256, torch.float32, torch.float32)
    x[1] *= 1e25
    out = _run(x, w, b, dy)
    assert out["rstd"][1] == 0 and np.array_equal(out["y"][1], _f64(b)) and np.isfinite(out["y"]).all()


def test_bad_rows_stay_alone():
    import torch
    x, w, b, dy = _make(40, 384, torch.bfloat16, torch.bfloat16)
    clean = _run(x, w, b, dy)
    x2 = x.clone()
    x2[3, 5], x2[17, 0] = float("nan"), float("inf")
    out = _run(x2, w, b, dy)
    rows = np.array([i for i in range(40) if i not in (3, 17)])
    assert np.isnan(out["y"][[3, 17]]).all()
    assert np.array_equal(out["y"][rows], clean["y"][rows]) and np.array_equal(out["dx"][rows], clean["dx"][rows])


def test_no_rows():
    import torch
    x, w, b, dy = _make(0, 96, torch.bfloat16, torch.float32)
    out = _run(x, w, b, dy)
    assert (out["dgamma"] == 0).all() and (out["dbeta"] == 0).all()


def test_in_place():
    import torch
    from mixture_experts_layer_18_gb300.training import LayerNorm
    x, w, b, dy = _make(300, 2048, torch.bfloat16, torch.bfloat16)
    ref = _run(x, w, b, dy)
    n = LayerNorm(300, 2048)
    y, dx = x.clone(), dy.clone()
    n.forward(y, w, b, y)
    n.backward(dx, x, w, dx)
    torch.cuda.synchronize()
    assert np.array_equal(_f64(y), ref["y"]) and np.array_equal(_f64(dx), ref["dx"])


def test_gradient_is_the_difference():
    """<dx, d> against the central difference of the definition along d."""
    import torch
    x, w, b, dy = _make(20, 200, torch.float32, torch.float32)
    out = _run(x, w, b, dy)
    X, D = _f64(x), _f64(dy)
    d = np.random.default_rng(0).standard_normal(X.shape)
    f = lambda v: (O.layer_norm(v, _f64(w), _f64(b), EPS)[0] * D).sum()  # noqa: E731
    h = 1e-5
    want = (f(X + h * d) - f(X - h * d)) / (2 * h)
    # every dx is within 64 * 8 U of rstd * |dy|-sized numbers; 4000 of them, of random signs, are summed
    tol = 512 * U * np.sqrt((np.abs(D) * np.abs(d)).sum() * np.abs(D).max() * np.abs(d).max()) * 4 + 1e-6
    assert abs((out["dx"] * d).sum() - want) <= tol


def test_same_results_every_run_and_on_a_side_stream():
    import torch
    x, w, b, dy = _make(5000, 1536, torch.bfloat16, torch.float32)
    first = _run(x, w, b, dy)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = _run(x, w, b, dy)
    for k in first:
        assert np.array_equal(first[k], second[k]), k


def test_captured_in_a_graph():
    import torch
    from mixture_experts_layer_18_gb300.training import LayerNorm
    x, w, b, dy = _make(256, 1024, torch.bfloat16, torch.bfloat16)
    ref = _run(x, w, b, dy)
    n = LayerNorm(256, 1024)
    io = n.empty_io()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n.forward(x, w, b, io["y"])
        n.backward(dy, x, w, io["dx"], io["dgamma"], io["dbeta"])
    g.replay()
    torch.cuda.synchronize()
    for k in io:
        assert np.array_equal(_f64(io[k]), ref[k]), k


def test_refused_tensors():
    import torch
    from mixture_experts_layer_18_gb300 import MoEError
    from mixture_experts_layer_18_gb300.training import LayerNorm
    x, w, b, dy = _make(8, 64, torch.bfloat16, torch.bfloat16)
    n = LayerNorm(8, 64)
    y = torch.empty_like(x)
    for bad in ((x.float(), w, b, y), (x[:4], w, b, y), (x, w.float(), b, y), (x, w, b[:3], y), (x, w, b, y.cpu()),
                (x.t().contiguous().t(), w, b, y), (x[:1].expand(8, 64), w, b, y)):
        with pytest.raises(MoEError):
            n.forward(*bad)
    with pytest.raises(MoEError):
        LayerNorm(8, 64, dtype=torch.float16)
    with pytest.raises(MoEError):
        LayerNorm(8, 64, backward=False).backward(dy, x, w, y)
