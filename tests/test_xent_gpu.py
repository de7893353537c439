"""Cross entropy over a vocabulary on the GPU against its float64 definition.

Tolerances.  The products of bf16 numbers are exact in fp32; a logit is a sum
of H of them, added in blocks of 16 into an fp32 accumulator, so its error is
below (H / 16 + 16) 2^-23 sum|x w| (E below, the largest of a row).  lse and
the loss move by as much, plus a few roundings of their own size.  A
probability's relative error is at most 2 E + 2^-20; dz is rounded to bf16
(8 significant bits: unit roundoff 2^-8) before the products, dX and dW once
after them."""
import numpy as np
import pytest

from oracle import training_oracle as O

pytestmark = pytest.mark.gpu

B8 = 2.0 ** -8
IGNORE = -100


def _f64(t):
    return t.double().cpu().numpy()


def _make(T, H, V, masked=0.0, seed=0, pad_x=0, pad_w=0, index="int64", sharp=2.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed * 7 + T + 31 * H + V)

    def rows(n, pad, scale):
        buf = torch.full((n, H + pad), 99.0, dtype=torch.bfloat16, device="cuda")
        v = buf[:, :H]
        v.copy_(torch.randn((n, H), generator=g, device="cuda") * scale)
        return v
    X, W = rows(T, pad_x, 1.0), rows(V, pad_w, sharp / H ** 0.5)
    t = torch.randint(0, V, (T,), generator=g, device="cuda").to(getattr(torch, index))
    if masked:
        t[torch.rand(T, generator=g, device="cuda") < masked] = IGNORE
    return X, W, t


def _run(X, W, t, dloss=None, reduction="mean", backward=True, op=None):
    import torch
    from mixture_experts_layer_18_gb300.training import CrossEntropy
    (T, H), V = X.shape, W.shape[0]
    c = op or CrossEntropy(T, H, V, ignore_index=IGNORE, index_dtype=t.dtype, backward=backward)
    c.ws.fill_(255)                                    # NaN patterns: nothing unwritten may be used
    c.forward(X, W, t)
    out = dict(loss=c.loss, lse=c.lse, total=c.total)
    if backward:
        io = c.empty_io()
        for v in io.values():
            v.fill_(7.0)
        c.ws.fill_(255)
        d = torch.ones(1, device="cuda") if dloss is None else dloss
        c.backward(X, W, t, d, io["dX"], io["dW"], reduction=reduction)
        out.update(io)
    torch.cuda.synchronize()
    out = {k: _f64(v) for k, v in out.items()}
    out["status"] = c.device_status()
    return out


def _logit_error(X, W):
    H = X.shape[1]
    return (H / 16 + 16) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T).max(1)


def _check(X, W, t, out, s=None, backward=True):
    """s: what reaches each row's loss (default: the mean's 1 / count)."""
    Xd, Wd, td = _f64(X), _f64(W), t.cpu().numpy()
    V = Wd.shape[0]
    loss, lse, mean = O.cross_entropy(Xd, Wd, td, IGNORE)
    on = O.counted(td, V, IGNORE)
    e = _logit_error(Xd, Wd) + 2.0 ** -21 * (1 + np.abs(lse))
    assert (np.abs(out["lse"] - lse) <= e).all(), np.abs(out["lse"] - lse).max()
    assert (np.abs(out["loss"] - loss) <= 2 * e * on).all(), np.abs(out["loss"] - loss).max()
    assert out["total"][2] == on.sum()
    assert abs(out["total"][1] - mean) <= 2 * e.max() and abs(out["total"][0] - loss.sum()) <= 2 * e.sum()
    if not backward:
        return
    if s is None:
        s = np.full(len(td), 1.0 / max(1, on.sum()))
    dX, dW, dz = O.cross_entropy_backward(Xd, Wd, td, s, IGNORE)
    p = np.exp(Xd @ Wd.T - lse[:, None]) * np.abs(s * on)[:, None]
    dev = B8 * np.abs(dz) + (2 * e[:, None] + 2.0 ** -20) * p      # error of dz
    n = 2.0 ** -20                                                 # accumulation of the products
    for name, ref, tol in (("dX", dX, dev @ np.abs(Wd) + n * (np.abs(dz) @ np.abs(Wd))),
                           ("dW", dW, dev.T @ np.abs(Xd) + n * (np.abs(dz).T @ np.abs(Xd)))):
        err = np.abs(out[name] - ref)
        assert (err <= B8 * np.abs(ref) + 1.01 * tol + 1e-38).all(), (name, err.max())


# one token, one entry; sizes around a tile (256) and a K block (64); odd
# everything; enough tiles for several rounds; slices of the vocabulary
SHAPES = [(1, 8, 1), (1, 64, 1000), (2, 72, 3), (7, 256, 32000), (128, 64, 256), (129, 128, 257), (255, 520, 511),
          (256, 64, 255), (257, 192, 5003), (1001, 1032, 2007), (600, 2048, 1537), (33, 4096, 700), (3000, 264, 4111),
          # the kernel for few tokens: both its widths, vocabularies around its 16 rows, long and short K
          (8, 1032, 15), (9, 40, 17), (16, 2056, 4999), (16, 8, 33), (5, 12000, 130), (16, 4096, 515)]


@pytest.mark.parametrize("T,H,V", SHAPES)
def test_cross_entropy_matches_definition(T, H, V):
    X, W, t = _make(T, H, V)
    out = _run(X, W, t)
    assert out["status"] == 0
    _check(X, W, t, out)


@pytest.mark.parametrize("masked", [0.3, 1.0])
@pytest.mark.parametrize("index", ["int32", "int64"])
def test_masked_rows(masked, index):
    X, W, t = _make(300, 128, 900, masked=masked, index=index)
    out = _run(X, W, t)
    _check(X, W, t, out)
    off = t.cpu().numpy() == IGNORE
    assert (out["loss"][off] == 0).all() and (out["dX"][off] == 0).all()
    if masked == 1.0:
        assert (out["total"] == 0).all() and not out["dW"].any()


@pytest.mark.parametrize("pad_x,pad_w", [(8, 0), (0, 24), (64, 8)])
def test_strided_rows(pad_x, pad_w):
    X, W, t = _make(200, 136, 777, pad_x=pad_x, pad_w=pad_w)
    _check(X, W, t, _run(X, W, t))


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_reductions(reduction):
    import torch
    X, W, t = _make(150, 64, 333, masked=0.2)
    on = O.counted(t.cpu().numpy(), 333, IGNORE)
    if reduction == "none":
        d = torch.randn(150, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
        s = _f64(d)
    else:
        d = torch.tensor([-2.5], device="cuda")
        s = np.full(150, -2.5 / (on.sum() if reduction == "mean" else 1))
    _check(X, W, t, _run(X, W, t, dloss=d, reduction=reduction), s=s)


def test_target_outside_the_vocabulary_is_reported():
    import torch
    import mixture_experts_layer_18_gb300 as M
    for index in ("int32", "int64"):
        X, W, t = _make(70, 64, 500, index=index)
        t[3], t[40] = 500, -7
        if index == "int64":
            t[41] = (1 << 33) + 5                      # its low 32 bits are a valid column
        out = _run(X, W, t)
        assert out["status"] == M.MOE_ERR_BAD_INDEX
        _check(X, W, t, out)                           # such rows do not count
        assert out["total"][2] == (67 if index == "int64" else 68)


@pytest.mark.parametrize("T,H", [(16, 4096), (16, 4104), (200, 512), (200, 4096), (333, 4136), (200, 8192)])
def test_log_sums_are_not_biased(T, H):
    """A tensor-core accumulator truncates: added up in one of them, 4096
    products move lse by 2e-5, every row the same way.  Segments of at most 512
    columns bound that: 32 additions, each of at most half a unit of 2^-21 on
    average (the logits that make up lse are below 8 here), and no more than two
    units (2^-20) from the few roundings of lse itself."""
    X, W, t = _make(T, H, 5003)
    out = _run(X, W, t, backward=False)
    Xd, Wd, td = _f64(X), _f64(W), t.cpu().numpy()
    loss, lse, _ = O.cross_entropy(Xd, Wd, td, IGNORE)
    z = Xd @ Wd.T
    p = np.exp(z - lse[:, None])
    assert (p * np.abs(z)).sum(1).mean() < 8
    tol = 32 * 2.0 ** -22 + 2 * 2.0 ** -20
    assert abs((out["lse"] - lse).mean()) <= tol
    assert abs((out["loss"] - loss).mean()) <= tol


@pytest.mark.parametrize("T,H,V", [(1, 128, 1000), (1, 1032, 3001), (5, 512, 2000), (31, 264, 1500), (32, 512, 9000)])
@pytest.mark.parametrize("reduction", ["mean", "none"])
def test_few_tokens_round_their_gradients_once(T, H, V, reduction):
    """dz of up to 32 tokens is held to 16 bits, so dX and dW carry their own
    rounding to bf16 and nothing else of that size: the root mean square of it
    is at most 2^-7 / sqrt(12) of the values' (5% for the chance in a few
    hundred of them)."""
    import torch
    X, W, t = _make(T, H, V)
    d = torch.linspace(0.3, 1.7, T, device="cuda") if reduction == "none" else None
    out = _run(X, W, t, dloss=d, reduction=reduction)
    Xd, Wd, td = _f64(X), _f64(W), t.cpu().numpy()
    _, lse, _ = O.cross_entropy(Xd, Wd, td, IGNORE)
    dz = np.exp(Xd @ Wd.T - lse[:, None])
    dz[np.arange(T), td] -= 1
    dz *= np.full((T, 1), 1.0 / T) if d is None else _f64(d)[:, None]
    for got, want in ((out["dX"], dz @ Wd), (out["dW"], dz.T @ Xd)):
        assert np.linalg.norm(got - want) <= 1.05 * 2.0 ** -7 / 12 ** 0.5 * np.linalg.norm(want)


def test_large_logits():
    """Logits in the hundreds: exp of the raw logit would overflow."""
    X, W, t = _make(130, 256, 600, sharp=60.0)
    X *= 4
    out = _run(X, W, t)
    assert np.isfinite(out["loss"]).all() and np.abs(out["lse"]).max() > 400
    _check(X, W, t, out)


def test_bad_rows_stay_alone():
    X, W, t = _make(140, 64, 300)
    clean = _run(X, W, t)
    X2 = X.clone()
    X2[5, 3] = float("nan")
    t2 = t.clone()
    t2[5] = IGNORE                                     # ignored: its NaN reaches nothing
    out = _run(X2, W, t2)
    assert (out["loss"][5] == 0) and (out["dX"][5] == 0).all() and np.isfinite(out["dX"]).all()
    # (dW sums dz^T X over rows: 0 * NaN of the ignored row is the caller's NaN)
    rows = np.arange(140) != 5
    assert np.array_equal(out["loss"][rows], clean["loss"][rows])
    out = _run(X2, W, t)
    assert np.isnan(out["loss"][5]) and np.isfinite(out["loss"][rows]).all()
    assert np.isnan(out["dX"][5]).all() and np.array_equal(out["lse"][rows], clean["lse"][rows])


def test_bad_rows_stay_alone_among_few_tokens():
    X, W, t = _make(6, 72, 900)
    clean = _run(X, W, t, backward=False)
    X[2, 70], X[4, 0] = float("nan"), float("inf")
    out = _run(X, W, t, backward=False)
    assert np.isnan(out["loss"][[2, 4]]).all() and np.isnan(out["lse"][[2, 4]]).all()
    keep = [0, 1, 3, 5]
    assert np.array_equal(out["loss"][keep], clean["loss"][keep])
    assert np.array_equal(out["lse"][keep], clean["lse"][keep])


def test_ignored_value_inside_the_vocabulary():
    from mixture_experts_layer_18_gb300.training import CrossEntropy
    for T in (12, 130):
        X, W, t = _make(T, 64, 300)
        t[::3] = 7
        c = CrossEntropy(T, 64, 300, ignore_index=7)
        out = _run(X, W, t, op=c)
        ref, _, mean = O.cross_entropy(_f64(X), _f64(W), t.cpu().numpy(), 7)
        assert (out["loss"][::3] == 0).all() and abs(out["total"][1] - mean) <= 1e-4 * mean
        assert out["total"][2] == (ref != 0).sum()


def test_no_tokens():
    X, W, t = _make(0, 64, 300)
    out = _run(X, W, t)
    assert (out["total"] == 0).all() and not out["dW"].any() and out["dX"].size == 0


def test_one_output_alone():
    import torch
    from mixture_experts_layer_18_gb300.training import CrossEntropy
    X, W, t = _make(300, 200, 1000)
    both = _run(X, W, t)
    c = CrossEntropy(300, 200, 1000)
    io = c.empty_io()
    one = torch.ones(1, device="cuda")
    c.forward(X, W, t)
    c.backward(X, W, t, one, io["dX"], None)
    c.backward(X, W, t, one, None, io["dW"])
    torch.cuda.synchronize()
    assert np.array_equal(_f64(io["dX"]), both["dX"]) and np.array_equal(_f64(io["dW"]), both["dW"])


def test_several_pieces_of_the_vocabulary():
    """So many tokens that the vocabulary takes three pieces, the last of them
    ragged (the reference runs in 64 bits on the GPU, by rows)."""
    import torch
    T, H, V = 40001, 64, 9001
    X, W, t = _make(T, H, V, masked=0.1)
    out = _run(X, W, t)
    assert out["status"] == 0
    Xd, Wd = X.double(), W.double()
    on = t >= 0
    s = 1.0 / float(on.sum())
    dX, dW = torch.zeros_like(Xd), torch.zeros_like(Wd)
    aX, aW = torch.zeros_like(Xd), torch.zeros_like(Wd)
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    for i in range(0, T, 8000):
        x, k, q = Xd[i:i + 8000], t[i:i + 8000].clamp(min=0), on[i:i + 8000, None]
        lp = torch.log_softmax(x @ Wd.T, 1)
        loss[i:i + 8000] = torch.where(q[:, 0], -lp.gather(1, k[:, None])[:, 0], 0.0)
        dz = lp.exp().scatter_add(1, k[:, None], -torch.ones_like(k[:, None], dtype=torch.float64))
        dz = torch.where(q, dz * s, 0.0)
        dX[i:i + 8000], aX[i:i + 8000] = dz @ Wd, dz.abs() @ Wd.abs()
        dW += dz.T @ x
        aW += dz.abs().T @ x.abs()
    e = (H / 16 + 16) * 2.0 ** -23 * float((Xd.abs().sum(1).max() * Wd.abs().max()))
    assert np.abs(out["loss"] - _f64(loss)).max() <= 2 * e + 2.0 ** -18
    for name, ref, a in (("dX", dX, aX), ("dW", dW, aW)):
        # |p| <= |dz| away from the target; at the target 1 - p carries p's error
        tol = B8 * ref.abs() + (B8 + 4 * e + 2.0 ** -18) * a + 2 * (2 * e + 2.0 ** -20) * s * (
            Wd.abs().max() if name == "dX" else Xd.abs().sum(0).max())
        err = (torch.from_numpy(out[name]).cuda() - ref).abs()
        assert (err <= tol).all(), (name, float(err.max()))


def test_gradient_is_the_difference():
    """<dX, d> and <dW, e> against central differences of the definition."""
    X, W, t = _make(40, 96, 250, masked=0.1)
    out = _run(X, W, t)
    Xd, Wd, td = _f64(X), _f64(W), t.cpu().numpy()
    rng = np.random.default_rng(0)
    h = 1e-5
    for name, at in (("dX", 0), ("dW", 1)):
        d = rng.standard_normal((Xd, Wd)[at].shape)
        f = lambda u: O.cross_entropy(*((Xd + u * d, Wd) if at == 0 else (Xd, Wd + u * d)), td, IGNORE)[2]  # noqa: E731
        want = (f(h) - f(-h)) / (2 * h)
        # two bf16 roundings (of dz, of the result) of terms with independent signs
        tol = 6 * 2 * B8 * np.sqrt(((out[name] * d) ** 2).sum()) + 1e-7
        assert abs((out[name] * d).sum() - want) <= tol, name


def test_same_results_every_run_and_on_a_side_stream():
    import torch
    X, W, t = _make(900, 264, 3001, masked=0.2)
    first = _run(X, W, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = _run(X, W, t)
    for k in first:
        assert np.array_equal(first[k], second[k]), k


def test_captured_in_a_graph():
    import torch
    from mixture_experts_layer_18_gb300.training import CrossEntropy
    X, W, t = _make(300, 128, 2000)
    ref = _run(X, W, t)
    c = CrossEntropy(300, 128, 2000)
    io = c.empty_io()
    one = torch.ones(1, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.forward(X, W, t)
        c.backward(X, W, t, one, io["dX"], io["dW"])
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(_f64(c.loss), ref["loss"])
    for k in io:
        assert np.array_equal(_f64(io[k]), ref[k]), k


def test_refused_tensors():
    import torch
    from mixture_experts_layer_18_gb300 import MoEError
    from mixture_experts_layer_18_gb300.training import CrossEntropy
    X, W, t = _make(16, 64, 100)
    c = CrossEntropy(16, 64, 100)
    one = torch.ones(1, device="cuda")
    for bad in ((X.float(), W, t), (X[:8], W, t), (X, W[:50], t), (X, W, t.int()), (X, W, t[:4]), (X, W.cpu(), t)):
        with pytest.raises(MoEError):
            c.forward(*bad)
    c.forward(X, W, t)
    for kw in (dict(reduction="most"), dict(reduction="none")):
        with pytest.raises(MoEError):
            c.backward(X, W, t, one, None, None, **kw)
    with pytest.raises(MoEError):
        CrossEntropy(16, 60, 100)
    with pytest.raises(MoEError):
        CrossEntropy(16, 64, 100, backward=False).backward(X, W, t, one, None, None)
