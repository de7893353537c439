"""MoELayer's Python side on host tensors."""
import gc
import subprocess
import sys
import weakref

import numpy as np
import pytest
import torch

from conftest import ROOT
from mixture_experts_layer_18_gb300 import MOE_ERR_INVALID_ARG, MoEError, layer, training


@pytest.fixture
def L():
    return layer.MoELayer(4, 64, 4, 64, 2, device="cpu")


VIEWS = ("x_perm", "h13", "act")


def test_views_follow_the_buffer(L):
    """`saved` replaced, or its memory: the views lie in what the library is given."""
    def lies_in(buffer):
        at = buffer.data_ptr()
        return [getattr(L, n).data_ptr() - at for n in VIEWS] == [getattr(L.layout, n) for n in VIEWS]
    assert lies_in(L.saved)
    L.saved.data = torch.empty(L.layout.total, dtype=torch.uint8)
    assert lies_in(L.saved)
    L.saved = torch.empty(L.layout.total + 16, dtype=torch.uint8)
    assert lies_in(L.saved)


def test_a_view_is_the_readers_own(L):
    for n in VIEWS:
        shape = getattr(L, n).shape
        getattr(L, n).t_()
        assert getattr(L, n).shape == shape


def test_views_hold_no_memory(L):
    """A replaced buffer is freed without another look at the views."""
    for replace in (lambda b: setattr(L, "saved", b), lambda b: setattr(L.saved, "data", b)):
        memory = np.empty(L.layout.total, np.uint8)
        gone = weakref.ref(memory)
        L.saved = torch.from_numpy(memory)
        del memory
        for n in VIEWS:
            getattr(L, n)
        replace(torch.empty(L.layout.total, dtype=torch.uint8))
        gc.collect()
        assert gone() is None


def test_views_after_other_ways_to_replace_the_memory(L):
    """By a reference taken before, by size alone, in place; and without a buffer."""
    buffer = L.saved
    for n in VIEWS:
        getattr(L, n)
    buffer.data = torch.empty(L.layout.total, dtype=torch.uint8)
    assert L.h13.data_ptr() == buffer.data_ptr() + L.layout.h13
    buffer.data = buffer.data[:L.layout.act]
    assert L.h13.data_ptr() == buffer.data_ptr() + L.layout.h13
    with pytest.raises(RuntimeError):
        L.act
    del L.saved, buffer
    with pytest.raises(AttributeError):
        L.h13
    L.saved = torch.zeros(L.layout.total, dtype=torch.uint8)
    assert not L.h13.any()


def test_views_seen_in_inference_mode_first(L):
    """They do not make later ones inference tensors, which could not be written."""
    with torch.inference_mode():
        for n in VIEWS:
            getattr(L, n)
    for n in VIEWS:
        getattr(L, n).fill_(1)
    assert not L.h13.is_inference() and L.h13.eq(1).all()


def test_views_share_the_buffer_and_nothing_else(L):
    for n in VIEWS:
        a, b = getattr(L, n), getattr(L, n)
        a.fill_(2)
        assert b.eq(2).all() and b._version == a._version == L.saved._version
        a.requires_grad_()
        assert not b.requires_grad and not getattr(L, n).requires_grad


def test_import_needs_no_cuda_in_torch():
    """A torch built without CUDA lacks these two; its own message comes at the first call."""
    code = ("import torch; del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream\n"
            "from mixture_experts_layer_18_gb300 import layer, training\n"
            "assert training._current_device is layer._current_device is torch.cuda.current_device\n"
            "assert callable(layer._current_stream) and training._current_stream is layer._current_stream\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.fixture
def calls(L, monkeypatch):
    """L with a library that does nothing; the names of the calls that reach it."""
    seen = []
    for name in ("moe_forward", "moe_checkpoint_save", "moe_checkpoint_restore"):
        monkeypatch.setattr(layer, name, lambda *a, name=name: seen.append(name) or 0)
    monkeypatch.setattr(layer, "_stream", lambda s: 0)
    monkeypatch.setattr(layer, "_current_device", lambda: None)

    def device(self, _):
        self.index, self.device = -1, torch.device("cpu")
    monkeypatch.setattr(training._Op, "_device", device)
    return seen


def test_save_needs_the_forwards_h13(L, calls):
    """After a forward that kept none, an earlier one's would go into the checkpoint."""
    ck, X = L.checkpoint(), torch.zeros((4, 64), dtype=torch.bfloat16)

    def refused():
        calls.clear()
        with pytest.raises(MoEError) as e:
            L.save(ck, X)
        return e.value.code == MOE_ERR_INVALID_ARG and not calls

    def forward(save):
        L.forward(X, X, X, X, save=save)
    L.save(ck, X)                                # (what the caller wrote itself)
    buffer, h13 = L.saved, L.h13
    for again in (lambda: forward(True), lambda: forward(None), lambda: L.restore(ck), lambda: h13.fill_(1),
                  lambda: buffer[L.layout.h13:L.layout.act].zero_(), lambda: L.h13, lambda: L.saved,
                  lambda: setattr(buffer, "data", torch.empty(L.layout.total, dtype=torch.uint8)),
                  lambda: setattr(L, "saved", torch.empty(L.layout.total, dtype=torch.uint8))):
        forward(True)
        L.save(ck, X)
        forward(False)
        assert refused() and refused()
        again()
        calls.clear()
        L.save(ck, X)
        assert calls == ["moe_checkpoint_save"]


def test_save_after_captured_forwards(L, calls, monkeypatch):
    """A captured call changes nothing yet; once one that keeps h13 has been captured, its replays may
    have come after any other call."""
    ck, X, capturing = L.checkpoint(), torch.zeros((4, 64), dtype=torch.bfloat16), [False]
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])

    def forward(save, captured=False):
        capturing[0] = captured
        L.forward(X, X, X, X, save=save)
        capturing[0] = False
    forward(True)
    forward(False, captured=True)
    L.save(ck, X)
    forward(False)
    with pytest.raises(MoEError):
        L.save(ck, X)
    forward(True, captured=True)
    L.save(ck, X)
    forward(False)
    L.save(ck, X)


def test_save_after_forwards_on_other_streams(L, calls, monkeypatch):
    """Which may be captured although the current one is not, or about which torch cannot tell."""
    class Stream:
        cuda_stream = 7
    ck, X, current = L.checkpoint(), torch.zeros((4, 64), dtype=torch.bfloat16), [7]
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(layer, "_current_stream", lambda device: current[0])

    def cannot_tell():
        raise RuntimeError("a blocking stream is being captured")

    def refused():
        try:
            L.save(ck, X)
        except MoEError:
            return True
        return False
    L.forward(X, X, X, X, stream=Stream, save=False)
    assert refused()
    L.forward(X, X, X, X, stream=Stream)
    current[0] = 8
    L.forward(X, X, X, X, stream=Stream, save=False)
    assert not refused()
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", cannot_tell)
    L.forward(X, X, X, X, save=False)
    assert not refused()
    L.forward(X, X, X, X)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    L.forward(X, X, X, X, save=False)
    assert not refused()
