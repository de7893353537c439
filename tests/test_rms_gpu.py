"""The RMS norm with residual and MXFP8 output on the GPU against its float64
definition, and MXFP8 rows read back.

Tolerances.  U = 2^-24 is the unit roundoff of fp32; a stored type adds its own
(2^-8 for bf16).  A row's sum of squares is a tree of at most 64 additions of
positive numbers, off by 66 U; rstd by half of that and 3 U: E = 36 U.  With the
residual's addition (U) and the products (3 U) a value of y is off by 40 U.  Codes
lie between those of y (1 - 40 U) and y (1 + 40 U).  dx is the definition's at the
h and rstd that the backward reads: its one sum is off by (66 + 4) U of the sum of
the magnitudes.  A column's sum over T rows is off by (64 + T / 32) U of the sum
of its magnitudes."""
import numpy as np
import pytest

from oracle import moe_oracle as M
from oracle import training_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
Y_ERR = 40 * U
EPS = 1e-6


def _stored(dtype):
    import torch
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def _f64(t):
    return None if t is None else t.double().cpu().numpy()


def _rows(T, H, dtype, g, pad=0, off=0, scale=1.5):
    import torch
    buf = torch.full((T, H + pad + off), 1e4, dtype=dtype, device="cuda")
    v = buf[:, off:off + H]
    v.copy_(torch.randn((T, H), generator=g, device="cuda") * scale)
    return v


def _make(T, H, dtype, wdtype, pad=0, off=0, residual=True):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + H)
    x, dy, dh = (_rows(T, H, dtype, g, pad, off) for _ in range(3))
    r = _rows(T, H, dtype, g, pad, off, 0.7) if residual else None
    return x, r, (1 + 0.3 * torch.randn(H, generator=g, device="cuda")).to(wdtype), dy, dh


def _check_codes(mx, y):
    """The codes of y [T, H] (float64), each within what y's error allows."""
    T, H = y.shape
    lo, hi = np.abs(y) * (1 - Y_ERR), np.abs(y) * (1 + Y_ERR)
    block = lambda v: v.reshape(T, H // 32, 32)      # noqa: E731
    sb = mx.scales.cpu().numpy().astype(np.int64)
    e = [M.mx_block_exponent(block(v).max(2)) + 127 for v in (lo, hi)]
    assert ((sb == e[0]) | (sb == e[1])).all()
    s = np.ldexp(1.0, sb - 127)[:, :, None]
    q = M.e4m3_decode(mx.codes.cpu().numpy())
    a, b = (M.e4m3_round(block(v) / s).reshape(T, H) for v in (lo, hi))
    assert ((np.abs(q) >= a) & (np.abs(q) <= b)).all()
    assert (np.where(np.abs(q) > 0, np.signbit(q) == np.signbit(y), True)).all()


def _check(x, r, w, dy, dh, eps=EPS, mx=False, outputs=("h", "y"), inplace=False):
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows, RMSNorm
    T, H = x.shape
    n = RMSNorm(T, H, dtype=x.dtype, weight_dtype=x.dtype if w is None else w.dtype, eps=eps)
    X, R = _f64(x), _f64(r)
    h, y, rstd = O.rms_norm(X, R, _f64(w), eps)
    io = n.empty_io()
    for t in io.values():
        t.fill_(7.0)
    if inplace:
        io["h"], io["y"] = r, x
    enc = MXRows(T, H) if mx else None
    n.forward(x, w, io["y"] if "y" in outputs else None, residual=r, h=io["h"] if r is not None else None, encoded=enc)
    torch.cuda.synchronize()
    ux = _stored(x.dtype)
    if "y" in outputs:
        assert (np.abs(_f64(io["y"]) - y) <= ux * np.abs(y) + (1 + ux) * Y_ERR * np.abs(y)).all()
    else:
        assert (io["y"] == 7.0).all()
    if r is not None:
        # (a rounding of the sum to fp32 first, where that is not exact)
        assert (np.abs(_f64(io["h"]) - h) <= (ux + U) * np.abs(h)).all()
    assert (np.abs(_f64(n.rstd) - rstd) <= 36 * U * rstd).all()
    if mx:
        _check_codes(enc, y)
        for dt in (torch.float32, torch.bfloat16):
            out = torch.full((T, H + 5), 3.0, dtype=dt, device="cuda")
            enc.decode(out[:, :H])
            want = M.dequantize_mxfp8(enc.codes.cpu().numpy(), enc.scales.cpu().numpy(), 1)
            assert np.array_equal(_f64(out[:, :H]), want) and (out[:, H:] == 3.0).all()
    if dy is None:
        return
    hs = io["h"] if r is not None else x
    rs = _f64(n.rstd)
    D, G, Hs, DH = _f64(dy), 1.0 if w is None else _f64(w), _f64(hs), _f64(dh)
    dx, dg = O.rms_norm_backward(D, Hs, None if w is None else G, rs, DH)
    n.backward(dy, hs, w, io["dx"], io["dgamma"], dh=dh)
    torch.cuda.synchronize()
    xh, g = np.abs(Hs) * rs[:, None], np.abs(D * G)
    size = rs[:, None] * (g + xh * (g * xh).mean(1)[:, None]) + (0 if DH is None else np.abs(DH))
    assert (np.abs(_f64(io["dx"]) - dx) <= ux * np.abs(dx) + (1 + ux) * 75 * U * size).all()
    uw = _stored(io["dgamma"].dtype)
    tol = uw * np.abs(dg) + (1 + uw) * (66 + T / 32) * U * (np.abs(D) * xh).sum(0)
    assert (np.abs(_f64(io["dgamma"]) - dg) <= tol).all()


# every width class of the fused kernels and the long rows past them
SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (33, 64), (129, 96), (1000, 256), (257, 264), (700, 513), (311, 1000),
          (130, 1536), (400, 2049), (90, 2560), (70, 3584), (640, 4096), (97, 4104), (70, 5001), (65, 8192), (40, 8200),
          (33, 16384), (9, 16392), (5, 20001), (200, 9001), (31, 12004), (17, 16377)]


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16/f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_rms_norm_matches_definition(T, H, kind, residual):
    import torch
    dt = torch.float32 if kind == "f32" else torch.bfloat16
    wt = torch.bfloat16 if kind == "bf16" else torch.float32
    x, r, w, dy, dh = _make(T, H, dt, wt, residual=residual)
    _check(x, r, w, dy, dh if residual else None, mx=H % 32 == 0)


@pytest.mark.parametrize("pad,off", [(8, 0), (24, 8), (7, 0), (5, 3)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("H", [544, 4096, 20000])
def test_strided_rows(pad, off, dtype, H):
    import torch
    dt = getattr(torch, dtype)
    x, r, w, dy, dh = _make(130 if H < 9000 else 7, H, dt, dt, pad, off)
    _check(x, r, w, dy, dh, mx=True)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("H", [300, 320, 20000])
def test_tensors_at_different_offsets(dtype, H):
    import torch
    dt = getattr(torch, dtype)
    x, r, w, dy, dh = _make(23, H, dt, torch.float32, pad=3)
    r = r.contiguous()
    dh = torch.nn.functional.pad(dh, (1, 0))[:, 1:]
    _check(x, r, w, dy, dh, mx=H % 32 == 0)


@pytest.mark.parametrize("T,H", [(77, 512), (77, 515), (9, 20000), (9, 20001), (40, 12000)])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_in_place(T, H, dtype):
    """h over the residual, y over x; dx over each of its inputs."""
    import torch
    from mixture_experts_layer_18_gb300.training import RMSNorm
    dt = getattr(torch, dtype)
    x, r, w, dy, dh = _make(T, H, dt, dt)
    n = RMSNorm(T, H, dtype=dt)
    io = n.empty_io()
    n.forward(x, w, io["y"], residual=r, h=io["h"])
    n.backward(dy, io["h"], w, io["dx"], io["dgamma"], dh=dh)
    for name in ("dy", "h", "dh"):
        a = dict(dy=dy.clone(), h=io["h"].clone(), dh=dh.clone())
        dg = torch.empty_like(io["dgamma"])
        n.backward(a["dy"], a["h"], w, a[name], dg, dh=a["dh"])
        assert torch.equal(a[name], io["dx"]) and torch.equal(dg, io["dgamma"]), name
    _check(x.clone(), r.clone(), w, None, None, inplace=True)
    xs, rs = x.clone(), r.clone()
    n.forward(xs, w, rs, residual=rs, h=xs)
    assert torch.equal(xs, io["h"]) and torch.equal(rs, io["y"])


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_many_rows_and_codes_alone(dtype):
    import torch
    dt = getattr(torch, dtype)
    x, r, w, dy, dh = _make(20011, 192, dt, torch.float32)
    _check(x, r, w, dy, dh, mx=True)
    _check(x, None, w, None, None, mx=True, outputs=())
    _check(x, r, None, dy, None, mx=True, outputs=())


def test_bad_rows_stay_rows_of_their_own():
    """NaN, infinity, zeros (with eps 0 too), rows whose squares leave fp32 and
    tiny rows, among ordinary ones."""
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows, RMSNorm
    g = torch.Generator(device="cuda").manual_seed(1)
    for dt in (torch.float32, torch.bfloat16):
        x = torch.randn((40, 256), generator=g, device="cuda").to(dt)
        clean = x.clone()
        x[3, 7], x[5, 9], x[8], x[11], x[13] = float("nan"), float("inf"), 0.0, 1e30, x[13] * 1e-30
        n, n2 = RMSNorm(40, 256, dtype=dt), RMSNorm(40, 256, dtype=dt)
        y, y2, m, m2 = torch.empty_like(x), torch.empty_like(x), MXRows(40, 256), MXRows(40, 256)
        n.forward(x, None, y, encoded=m)
        n2.forward(clean, None, y2, encoded=m2)
        ok = [i for i in range(40) if i not in (3, 5, 8, 11, 13)]
        assert torch.equal(y[ok], y2[ok]) and torch.equal(m.codes[ok], m2.codes[ok])
        assert torch.equal(m.scales[ok], m2.scales[ok])
        assert y[3].isnan().all() and y[5, 9].isnan() and not y[8].any() and not y[11].any()
        assert not m.codes[8].any() and not m.scales[8].any()
        want = x[13].double() / (x[13].double().square().mean() + 1e-6).sqrt()
        assert (y[13].double() - want).abs().max() <= 2.0 ** -7 * want.abs().max()
        z = RMSNorm(40, 256, dtype=dt, eps=0.0)
        z.forward(torch.zeros_like(x), None, y)
        assert y.isnan().all()                                  # 0 / 0, as the formula has it


def test_tiny_values_have_codes():
    """Blocks below the smallest scale, and values of a thousand binades."""
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows
    rng = np.random.default_rng(0)
    x = np.ldexp(rng.standard_normal((64, 96)), rng.integers(-130, 120, (64, 96))).astype(np.float32)
    x[:8] = np.ldexp(rng.standard_normal((8, 96)), -124)
    x = torch.from_numpy(x).cuda().bfloat16()
    m = MXRows(64, 96)
    m.encode(x)
    codes, scales = M.quantize_mxfp8(_f64(x), 1)
    assert np.array_equal(m.codes.cpu().numpy(), codes) and np.array_equal(m.scales.cpu().numpy(), scales)
    out = torch.empty((64, 96), device="cuda")
    m.decode(out)
    assert np.array_equal(_f64(out), M.dequantize_mxfp8(codes, scales, 1))
    b = torch.empty((64, 96), dtype=torch.bfloat16, device="cuda")
    m.decode(b)
    assert torch.equal(b, out.bfloat16())


def test_every_code_is_read_back():
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows
    m = MXRows(256, 256)
    m.codes.copy_(torch.arange(256, dtype=torch.uint8)[None, :].expand(256, 256))
    m.scales.copy_(torch.arange(256, dtype=torch.int32)[:, None].expand(256, 8).to(torch.uint8))
    m.scales[248:] = 120                                         # (scales that no block gets)
    out = torch.empty((256, 256), device="cuda")
    m.decode(out)
    with np.errstate(over="ignore"):     # (a block with an infinity has scale 2^120; 448 2^120 lies past fp32's 2^128)
        want = M.dequantize_mxfp8(m.codes.cpu().numpy(), m.scales.cpu().numpy(), 1).astype(np.float32)
    assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


def test_no_rows():
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows, RMSNorm
    n, x, m = RMSNorm(0, 64), torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda"), MXRows(0, 64)
    dg = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    n.forward(x, None, x.clone(), residual=x, h=x.clone(), encoded=m)
    m.encode(x)
    m.decode(x)
    n.backward(x, x, None, x, dg)
    assert not dg.any()


def test_captured_and_same_every_time():
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows, RMSNorm
    x, r, w, dy, dh = _make(3001, 1024, torch.bfloat16, torch.float32)
    n, m = RMSNorm(3001, 1024, weight_dtype=torch.float32), MXRows(3001, 1024)
    io = n.empty_io()

    def step():
        n.forward(x, w, io["y"], residual=r, h=io["h"], encoded=m)
        n.backward(dy, io["h"], w, io["dx"], io["dgamma"], dh=dh)
    step()
    torch.cuda.synchronize()
    first = [t.clone() for t in (*io.values(), m.codes, m.scales)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in io.values():
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (*io.values(), m.codes, m.scales)))
    x.mul_(2)
    r.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(io["h"], 2 * first[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    io["h"].zero_()
    s.wait_stream(torch.cuda.current_stream())
    n.forward(x, w, io["y"], residual=r, h=io["h"], encoded=m, stream=s)
    s.synchronize()
    assert torch.equal(io["h"], 2 * first[1])


def test_elements_past_32_bits():
    """More than 2^32 elements of rows and codes: the last rows are their own."""
    import torch
    from mixture_experts_layer_18_gb300.training import MXRows, RMSNorm
    T, H = 2_100_000, 2048
    g = torch.Generator(device="cuda").manual_seed(3)
    tail = torch.randn((64, H), generator=g, device="cuda").bfloat16()
    x = torch.ones((T, H), dtype=torch.bfloat16, device="cuda")
    x[-64:] = tail
    n, small, m, ms = RMSNorm(T, H), RMSNorm(64, H), MXRows(T, H), MXRows(64, H)
    y, ys = torch.empty_like(x), torch.empty_like(tail)
    n.forward(x, None, y, encoded=m)
    small.forward(tail, None, ys, encoded=ms)
    assert torch.equal(y[-64:], ys) and torch.equal(m.codes[-64:], ms.codes) and torch.equal(m.scales[-64:], ms.scales)
    assert (y[:-64:1000] == 1.0).all()
    back, bs = torch.empty_like(x), torch.empty_like(tail)
    m.decode(back)
    ms.decode(bs)
    assert torch.equal(back[-64:], bs)
    del back, m
    dx, dxs = torch.empty_like(x), torch.empty_like(tail)
    n.backward(y, x, None, dx)
    small.backward(ys, tail, None, dxs)
    assert torch.equal(dx[-64:], dxs)
