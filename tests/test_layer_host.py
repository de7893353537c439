"""MoELayer's Python side on host tensors."""
import gc
import subprocess
import sys
import weakref

import numpy as np
import pytest
import torch

from conftest import ROOT
from mixture_experts_layer_18_gb300 import layer


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


def test_import_needs_no_cuda_in_torch():
    """A torch built without CUDA lacks these two; its own message comes at the first call."""
    code = ("import torch; del torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream\n"
            "from mixture_experts_layer_18_gb300 import layer, training\n"
            "assert training._current_device is layer._current_device is torch.cuda.current_device\n"
            "assert callable(layer._current_stream) and training._current_stream is layer._current_stream\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
