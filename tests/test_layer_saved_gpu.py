"""The saved activations of a layer when their buffer is replaced, and checkpoints
after forwards that keep h13, that do not, and that were captured into a graph."""
import pytest

pytestmark = pytest.mark.gpu


def _layer(seed=0):
    import torch
    from mixture_experts_layer_18_gb300.layer import MoELayer
    T, H, E, I, k = 200, 128, 8, 64, 2
    g = torch.Generator(device="cuda").manual_seed(seed)
    L = MoELayer(T, H, E, I, k)
    X, W13, W2 = (torch.randn(s, generator=g, device="cuda").bfloat16() for s in ((T, H), (E, H, 2 * I), (E, I, H)))
    L.route(torch.randn((T, E), generator=g, device="cuda"))
    return L, X, W13, W2, torch.empty_like(X), int(L.padded_offsets[-1])


def test_views_show_what_the_forward_writes():
    """Into a buffer whose memory was replaced after a look at the views."""
    import torch
    L, X, W13, W2, Y, n = _layer()
    L.forward(X, W13, W2, Y)
    first = [t[:n].clone() for t in (L.x_perm, L.h13, L.act)]
    L.saved.data = torch.zeros_like(L.saved)
    L.forward(X, W13, W2, Y)
    for a, b in zip(first, (L.x_perm, L.h13, L.act)):
        assert torch.equal(a, b[:n])


def test_save_follows_the_forwards():
    import torch
    from mixture_experts_layer_18_gb300 import MoEError
    L, X, W13, W2, Y, n = _layer()
    ck, want = L.checkpoint(), L.checkpoint()
    L.forward(X, W13, W2, Y)
    L.save(want, X)
    L.forward(2 * X, W13, W2, Y, save=False)
    with pytest.raises(MoEError):
        L.save(ck, X)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward(X, W13, W2, Y)
    L.forward(2 * X, W13, W2, Y, save=False)
    L.h13.zero_()
    graph.replay()
    L.save(ck, X)
    assert torch.equal(ck.h13.codes, want.h13.codes) and torch.equal(ck.h13.scales, want.h13.scales)
    side = torch.cuda.Stream()
    L, X, W13, W2, Y, n = _layer()
    L.forward(X, W13, W2, Y, save=False)
    side.wait_stream(torch.cuda.current_stream())
    L.forward(X, W13, W2, Y, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    L.save(ck, X)
    assert torch.equal(ck.h13.codes, want.h13.codes) and torch.equal(ck.x.codes, want.x.codes)
