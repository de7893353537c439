"""The Python side of the training-step operators, run on the CPU: host tensors
stand in for device memory and a recorder for the library's calls, so what is
checked is what would be launched."""
import threading
import weakref

import pytest
import torch

import mixture_experts_layer_18_gb300 as M
from mixture_experts_layer_18_gb300 import training


@pytest.fixture
def host(monkeypatch):
    """Ops on host memory; returns the module."""
    def device(self, _):
        self.index, self.device = -1, torch.device("cpu")
    monkeypatch.setattr(training._Op, "_device", device)
    monkeypatch.setattr(training._Op, "_current", lambda self, stream: 0)
    return training


def _entries(array, count):
    return [(array[i].src, array[i].dst, array[i].n, array[i].type) for i in range(count)]


def test_gradients_that_move_are_found(host, monkeypatch):
    """A gradient whose memory was replaced or resized is read and written where
    it is at the time of the call, never where it was."""
    seen = []
    monkeypatch.setattr(host, "moe_clip_grads", lambda t, n, *a: seen.append(_entries(t, n)) or 0)
    monkeypatch.setattr(host, "moe_grad_norm", lambda t, n, *a: seen.append(_entries(t, n)) or 0)
    a, b, o = torch.zeros(10), torch.zeros(6, dtype=torch.bfloat16), torch.zeros(10)

    def want(first, out):
        return [(first.data_ptr(), out.data_ptr(), first.numel(), M.MOE_TYPE_F32),
                (b.data_ptr(), b.data_ptr(), 6, M.MOE_TYPE_BF16)]
    c = host.GradClip([a, b], out=[o, b])
    for call in (lambda: c.clip(1.0), c.measure):
        call()
        assert seen[-1] == want(a, o)
        keep = a.data                                  # (so that its address is not given out again)
        a.data = torch.ones(10)
        call()
        assert seen[-1] == want(a, o) and seen[-1][0][0] != keep.data_ptr()
        keep = o.data
        o.data = torch.ones(10)
        call()
        assert seen[-1] == want(a, o) and seen[-1][0][1] != keep.data_ptr()
    n = len(seen)
    keep = a.data
    a.resize_(100)                                     # more than its memory holds: moved
    with pytest.raises(M.MoEError):
        c.clip(1.0)                                    # its output no longer fits
    o.resize_(100)
    c.clip(1.0)
    assert len(seen) == n + 1 and seen[-1] == want(a, o) and seen[-1][0][2] == 100
    a.data = torch.ones(100, dtype=torch.float64)
    with pytest.raises(M.MoEError):
        c.clip(1.0)


def test_memory_of_the_list_stays(host, monkeypatch):
    """Between a change and the next call the listed memory is not given away."""
    a = torch.zeros(1000)
    c = host.GradClip([a])
    held = [weakref.ref(t) for t in c._listed[-1]]
    a.data = torch.empty(0)
    assert held[0]().numel() == 1000 and held[0]().data_ptr() != a.data_ptr()


def test_memory_whose_address_is_recorded_stays(host):
    """The results' names may be given to other tensors; the memory that the
    library was given stays."""
    for op, names in ((host.GradClip([torch.zeros(8)]), ("norm", "ws", "status")),
                      (host.CrossEntropy(4, 64, 100), ("loss", "lse", "total")),
                      (host.LayerNorm(4, 64), ("mean", "rstd"))):
        held = {k: weakref.ref(getattr(op, k)) for k in names}
        for k in names:
            setattr(op, k, None)
        assert all(r() is not None for r in held.values()), op


class _Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 77


def test_calls_on_another_device_are_refused(monkeypatch):
    """An op of one device is not launched while another is current, nor on
    another's stream: the library launches on the current device."""
    monkeypatch.setattr(training, "_current_stream", lambda index: 5)
    op = training._Op()
    op.index, op.device = 1, torch.device("cuda", 1)
    monkeypatch.setattr(training, "_current_device", lambda: 1, raising=False)
    assert op._current(None) == 5 and op._current(_Stream(1)) == 77
    with pytest.raises(M.MoEError):
        op._current(_Stream(0))
    monkeypatch.setattr(training, "_current_device", lambda: 0)
    for stream in (None, _Stream(0), _Stream(1)):
        with pytest.raises(M.MoEError):
            op._current(stream)


def _two_calls(first, second):
    """Runs both at once, each from a thread of its own."""
    errors = []

    def run(f):
        try:
            f()
        except BaseException as e:      # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=run, args=(f,)) for f in (first, second)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(20)
    assert not errors, errors


@pytest.mark.parametrize("op", ["norm", "xent"])
def test_calls_of_two_threads_keep_their_strides(host, monkeypatch, op):
    """Both calls are inside the library at the same time; each has the
    distances of its own rows."""
    meet, seen = threading.Barrier(2, timeout=10), {}

    def library(d, x, *a):
        meet.wait()                     # (both callers have described their rows)
        seen[x] = (d.ld_x, d.ld_y if op == "norm" else d.ld_w)
        return 0
    monkeypatch.setattr(host, "moe_layer_norm", library)
    monkeypatch.setattr(host, "moe_cross_entropy", library)
    make = lambda pad: torch.zeros((6, 64 + pad), dtype=torch.bfloat16)[:, :64]   # noqa: E731
    x, other = [make(8), make(24)], [make(16), make(40)]
    if op == "norm":
        n = host.LayerNorm(6, 64)
        calls = [lambda i=i: n.forward(x[i], None, None, other[i]) for i in (0, 1)]
    else:
        c, t = host.CrossEntropy(6, 64, 6), torch.zeros(6, dtype=torch.int64)
        calls = [lambda i=i: c.forward(x[i], other[i], t) for i in (0, 1)]
    _two_calls(*calls)
    assert seen == {x[0].data_ptr(): (72, 80), x[1].data_ptr(): (88, 104)}
    assert (n if op == "norm" else c).dims.T == 6


@pytest.mark.parametrize("make", [
    lambda m: m.LayerNorm((1 << 32) + 4, 64), lambda m: m.LayerNorm(4, (1 << 32) + 64), lambda m: m.LayerNorm(1 << 31, 8),
    lambda m: m.CrossEntropy((1 << 32) + 4, 64, 100), lambda m: m.CrossEntropy(4, (1 << 32) + 64, 100),
    lambda m: m.CrossEntropy(4, 64, (1 << 32) + 100), lambda m: m.CrossEntropy(4, 64, 100, ignore_index=1 << 32),
    lambda m: m.CrossEntropy(4, 64, 100, ignore_index=-(1 << 31) - 1)])
def test_numbers_past_32_bits_are_refused(host, make):
    """The library's sizes have 32 bits; what does not fit would be cut to its
    low ones (4 rows instead of 2^32 + 4, another value ignored)."""
    with pytest.raises(M.MoEError):
        make(host)


def test_the_ends_of_32_bits_are_taken(host):
    for ignore in (-(1 << 31), (1 << 31) - 1):
        assert host.CrossEntropy(4, 64, 100, ignore_index=ignore).dims.ignore_index == ignore


def test_gradient_of_a_scalar_loss(host, monkeypatch):
    """The gradient of the sum or mean has its shape, () or [1]; one per row is [T]."""
    seen = []
    monkeypatch.setattr(host, "moe_cross_entropy_backward", lambda *a: seen.append(a[6]) or 0)
    c = host.CrossEntropy(4, 64, 100)
    X, W = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((100, 64), dtype=torch.bfloat16)
    t, io = torch.zeros(4, dtype=torch.int64), c.empty_io()

    def call(d, reduction):
        c.backward(X, W, t, d, io["dX"], io["dW"], reduction=reduction)
    for d in (torch.ones(()), torch.ones(1)):
        for reduction in ("sum", "mean"):
            call(d, reduction)
            assert seen[-1] == d.data_ptr()
    call(torch.ones(4), "none")
    for d, reduction in ((torch.ones(4), "mean"), (torch.ones(()), "none"), (torch.ones((1, 1)), "sum"),
                         (torch.ones(()).double(), "mean")):
        with pytest.raises(M.MoEError):
            call(d, reduction)
    assert c.mean.shape == ()


def test_refusals_name_the_tensor(host):
    """What the library refuses by its address or its rows' distance is named."""
    c = host.CrossEntropy(4, 64, 100)
    b = dict(dtype=torch.bfloat16)
    X, W, t = torch.zeros((4, 64), **b), torch.zeros((100, 64), **b), torch.zeros(4, dtype=torch.int64)
    one = torch.ones(1)
    off = torch.zeros(100 * 64 + 64, **b)
    off = off[1:]
    odd = torch.zeros((100, 68), **b)[:, :64]
    shifted = off[:4 * 64].view(4, 64)
    assert shifted.data_ptr() % 16
    for name, call in (("X", lambda: c.forward(shifted, W, t)),
                       ("W", lambda: c.forward(X, off[:6400].view(100, 64), t)),
                       ("X", lambda: c.forward(odd[:4], W, t)), ("W", lambda: c.forward(X, odd, t)),
                       ("dX", lambda: c.backward(X, W, t, one, shifted, None)),
                       ("dW", lambda: c.backward(X, W, t, one, None, off[:6400].view(100, 64)))):
        with pytest.raises(M.MoEError, match=rf"\b{name}\b"):
            call()
