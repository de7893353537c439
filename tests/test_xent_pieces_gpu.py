"""The cross entropy's backward where the vocabulary takes several pieces and
dX's sums several slices of each, against float64 on the GPU.

Tolerances are those of test_xent_gpu.py (errors of a logit, of a probability,
of dz stored in bf16), with the products' accumulation at one truncation
(2^-23 of the sum of magnitudes) per 16 terms.  Norms are bounded too, which
would show a piece or a slice left out: a value rounded to bf16 is off by at
most 2^-7 / sqrt(12) of itself in the root mean square, dz once (its errors are
independent) and the result once; 10% for the chance in them."""
import pytest

pytestmark = pytest.mark.gpu

B8 = 2.0 ** -8
RMS = 2.0 ** -7 / 12 ** 0.5

# (T, H, V, first column of the last piece)
SIZES = [
    # the last piece has fewer K blocks than a whole one has slices: 4 for 10, 1 for 3, 1 for 5, 4 for 5, 2 for 152
    (4096, 256, 33000, 32768), (4096, 1024, 32800, 32768), (8192, 128, 16385, 16384), (8192, 128, 16600, 16384),
    (7, 64, 2097152 + 100, 2097152),
    # as many and more
    (8192, 128, 20001, 16384), (4096, 520, 70001, 65536)]


def _reference(X, W, t, s):
    """dX, dW and for each the bound's sums: (value, |dz| products, p products, sum of dz^2 |row|^2)."""
    import torch
    Xd, Wd = X.double(), W.double()
    wn, xn = (Wd * Wd).sum(1), (Xd * Xd).sum(1)
    H = X.shape[1]
    dX, aX, bX = (torch.zeros_like(Xd) for _ in range(3))
    dW, aW, bW = (torch.zeros_like(Wd) for _ in range(3))
    sX = sW = 0.0
    step = max(1, (1 << 27) // W.shape[0])
    for i in range(0, len(t), step):
        x, k = Xd[i:i + step], t[i:i + step]
        on = (k >= 0).double()[:, None]
        k = k.clamp(min=0)[:, None]
        z = x @ Wd.T
        e = (H / 16 + 16) * 2.0 ** -23 * (x.abs() @ Wd.abs().T).amax(1, keepdim=True)
        lse = torch.logsumexp(z, 1, keepdim=True)
        e = e + 2.0 ** -21 * (1 + lse.abs())
        p = (z - lse).exp_()
        dz = p.scatter_add(1, k, -torch.ones_like(k, dtype=torch.float64)) * (s * on)
        u = (2 * e + 2.0 ** -20) * p * (s * on)              # error of dz before it is stored
        dX[i:i + step], aX[i:i + step], bX[i:i + step] = dz @ Wd, dz.abs() @ Wd.abs(), u @ Wd.abs()
        dW += dz.T @ x
        aW += dz.abs().T @ x.abs()
        bW += u.T @ x.abs()
        q = dz * dz
        sX += float((q @ wn).sum())
        sW += float((q.T @ xn[i:i + step]).sum())
    return dict(dX=(dX, aX, bX, sX), dW=(dW, aW, bW, sW))


@pytest.mark.parametrize("T,H,V,last", SIZES)
def test_pieces_in_slices(T, H, V, last):
    import torch
    from mixture_experts_layer_18_gb300.training import CrossEntropy
    g = torch.Generator(device="cuda").manual_seed(T + H + V)
    X = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    W = (torch.randn((V, H), generator=g, device="cuda") * (2 / H ** 0.5)).bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    t[::2] = torch.randint(last, V, t[::2].shape, generator=g, device="cuda")   # half of them in the last piece
    t[::7] = -100
    c = CrossEntropy(T, H, V)
    io = c.empty_io()
    one = torch.ones(1, device="cuda")
    c.ws.fill_(255)
    c.forward(X, W, t)
    c.ws.fill_(255)
    c.backward(X, W, t, one, io["dX"], io["dW"])
    assert c.device_status() == 0
    alone = torch.empty_like(io["dX"])
    c.ws.fill_(255)
    c.backward(X, W, t, one, alone, None)
    assert c.device_status() == 0 and torch.equal(alone, io["dX"])
    ref = _reference(X, W, t, 1.0 / float(c.count))
    for name, terms in (("dX", V), ("dW", T)):
        want, a, b, q = ref[name]
        n = (terms / 16 + 16) * 2.0 ** -23
        err = (io[name].double() - want).abs()
        assert (err <= B8 * want.abs() + 1.01 * ((B8 + n) * a + b) + 1e-38).all(), (name, float(err.max()))
        assert float(err.norm()) <= 1.1 * RMS * (float(want.norm()) ** 2 + q) ** 0.5 + float((n * a + b).norm()), name
