"""Global gradient norm and clipping on the GPU against their float64
definition.

Tolerances: a thread's squares are summed in fp32, at most 32 terms to an
accumulator and each rounded once when squared, then almost exactly: the sum of
squares is within 40 * 2^-24 of its value, the norm within half of that plus
its own rounding.  A clipped value adds the division's, the product's and the
stored type's rounding."""
import numpy as np
import pytest

from oracle import training_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
NORM_TOL = 21 * U


def _f64(t):
    return t.double().cpu().numpy()


def _stored(t):
    import torch
    return 2.0 ** -8 if t.dtype == torch.bfloat16 else U


def _clip(grads, max_norm, out=None):
    import torch
    from mixture_experts_layer_18_gb300.training import GradClip
    c = GradClip(grads, out=out)
    c.clip(max_norm)
    torch.cuda.synchronize()
    return float(c.norm), c.device_status()


def _check(grads, max_norm):
    import torch
    from mixture_experts_layer_18_gb300.training import GradClip
    ref_n, ref = O.clip_grads([_f64(g) for g in grads], max_norm)
    m = GradClip(grads)
    m.measure()
    torch.cuda.synchronize()
    assert abs(float(m.norm) - ref_n) <= NORM_TOL * ref_n
    out = [torch.full_like(g, 9.0) for g in grads]
    before = [g.clone() for g in grads]
    n, st = _clip(grads, max_norm, out)
    assert st == 0 and n == float(m.norm)
    for g, k in zip(grads, before):
        assert torch.equal(g, k)                       # the sources are left alone
    for o, r in zip(out, ref):
        tol = (_stored(o) + NORM_TOL + 4 * U) * np.abs(r) + 1e-44
        assert (np.abs(_f64(o) - r) <= tol).all()
    _clip(grads, max_norm)                             # in place: the same values
    for g, o in zip(grads, out):
        assert torch.equal(g, o)


def _rand(n, dtype, seed, scale=1.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)


def _types():
    import torch
    return [torch.float32, torch.bfloat16]


@pytest.mark.parametrize("sizes", [[1], [5, 0, 1, 17], [2048, 2047, 2049], [100_003], [3] * 60, [33_000, 1, 70_001, 9],
                                   [3_000_001, 5, 12_345]])
@pytest.mark.parametrize("max_norm", [0.5, 1e6])
def test_clip_matches_definition(sizes, max_norm):
    ts = [_rand(n, _types()[i % 2], 100 * i + n, 10.0 ** (-(i % 3))) for i, n in enumerate(sizes)]
    _check(ts, max_norm)


def test_more_tensors_than_one_launch_takes():
    _check([_rand(1 + 37 * (i % 11), _types()[i % 3 == 0], i) for i in range(1100)], 2.0)


@pytest.mark.parametrize("off_in,off_out", [(1, 1), (3, 3), (1, 2), (0, 5)])
def test_unaligned_tensors(off_in, off_out):
    """Slices of a flat buffer, source and result at different offsets too."""
    import torch
    for dt in _types():
        a, b = _rand(50_011, dt, 5), torch.empty(50_020, dtype=dt, device="cuda")
        src, dst = a[off_in:off_in + 50_000], b[off_out:off_out + 50_000]
        n, _ = _clip([src], 1.0, [dst])
        rn, ref = O.clip_grads([_f64(src)], 1.0)
        assert abs(n - rn) <= NORM_TOL * rn
        assert (np.abs(_f64(dst) - ref[0]) <= (_stored(dst) + NORM_TOL + 4 * U) * np.abs(ref[0]) + 1e-44).all()


def test_nothing_to_clip():
    import torch
    from mixture_experts_layer_18_gb300.training import GradClip
    for grads in ([], [torch.empty(0, device="cuda")], [torch.zeros(1000, device="cuda")]):
        c = GradClip(grads)
        c.norm.fill_(5.0)
        c.clip(1.0)
        assert float(c.norm) == 0.0 and c.device_status() == 0
        c.norm.fill_(5.0)
        c.measure()
        assert float(c.norm) == 0.0
    g = torch.zeros(1000, device="cuda")
    g[3] = -2.0
    assert _clip([g], 0.0) == (2.0, 0)                 # a limit of zero clears the gradients
    assert not g.any()


@pytest.mark.parametrize("scale", [1e25, 3e37, 1e-25, 1e-38, 1e-42])
def test_squares_outside_fp32(scale):
    """Norms whose squares overflow or vanish in fp32 are still right."""
    for dt in _types():
        if scale < 1e-38 and dt != _types()[0]:
            continue
        g = _rand(7001, dt, 3) * 0.01 * scale
        n, st = _clip([g.clone(), _rand(9, dt, 4) * 0], 3e38)
        ref = O.grad_norm([_f64(g)])
        # a subnormal norm is a multiple of 2^-149
        assert st == 0 and abs(n - ref) <= NORM_TOL * ref + 2.0 ** -149


def test_norm_that_is_not_finite_is_reported():
    import torch
    import mixture_experts_layer_18_gb300 as M
    for v in (float("inf"), -float("inf"), float("nan"), 3e38):
        g = _rand(5000, torch.float32, 1)
        g[1234] = v
        if v == 3e38:
            g[:200] = v                                # finite values, a norm past fp32
        keep = g.clone()
        n, st = _clip([g], 1.0)
        assert st == M.MOE_ERR_BAD_INPUT and not np.isfinite(n)
        assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(keep))   # unscaled


def test_large_tensor_past_32_bits():
    """More than 2^32 elements in one tensor: 64-bit offsets."""
    import torch
    n = (1 << 32) + 4099
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[0], g[-1], g[1 << 31] = 3.0, 4.0, 12.0
    norm, st = _clip([g], 1.3)
    assert st == 0 and norm == 13.0
    got = [float(g[i]) for i in (0, n - 1, 1 << 31)]
    want = [float(torch.tensor(v * 0.1).bfloat16()) for v in (3.0, 4.0, 12.0)]
    assert np.allclose(got, want, rtol=2.0 ** -8)
    assert not g[1:1 << 31].any()


def test_same_norm_every_run_and_on_a_side_stream():
    import torch
    from mixture_experts_layer_18_gb300.training import GradClip
    gs = [_rand(1_000_003, _types()[i % 2], i) for i in range(9)]
    c = GradClip(gs)
    c.measure()
    first = float(c.norm)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            c.measure(stream=s)
            assert float(c.norm) == first


def test_captured_in_a_graph():
    import torch
    from mixture_experts_layer_18_gb300.training import GradClip
    gs = [_rand(70_001, t, 2) for t in _types()]
    out = [torch.empty_like(g) for g in gs]
    c = GradClip(gs, out=out)
    c.clip(0.7)
    ref = [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.clip(0.7)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_refused_lists():
    import torch
    from mixture_experts_layer_18_gb300 import MoEError
    from mixture_experts_layer_18_gb300.training import GradClip
    a = torch.zeros(8, 8, device="cuda")
    for grads, out in (([a.half()], None), ([a.t()[1:]], None), ([a], []), ([a], [a.bfloat16()]), ([a, a.cpu()], None)):
        with pytest.raises(MoEError):
            GradClip(grads, out=out)
    with pytest.raises(MoEError):
        GradClip([a]).clip(-1.0)
