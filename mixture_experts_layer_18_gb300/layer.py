"""Caller-side buffers for the C ABI, allocated with PyTorch.

PyTorch supplies device memory and the stream handle; every computation is a
call into libmoe_gb300.so through the binding in ``__init__``.  A ``MoELayer``
owns the routing arrays, the saved activations and the three workspaces of
one problem shape, and raises ``MoEError`` on any non-OK return code.
"""
from __future__ import annotations

import torch

from . import (MOE_BF16, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_F32, MOE_FP8_BWD, MOE_MXFP8,
               MOE_OK, MOE_WS_BACKWARD, MOE_WS_FORWARD, MOE_WS_ROUTE, MoEError, moe_backward,
               moe_checkpoint, moe_checkpoint_restore, moe_checkpoint_save, moe_dims, moe_forward,
               moe_max_rows, moe_route, moe_route_backward, moe_route_out, moe_saved_layout_of,
               moe_workspace_size)

MODES = {"f32": MOE_F32, "bf16": MOE_BF16, "mxfp8": MOE_MXFP8, "fp8_bwd": MOE_FP8_BWD}

# torch.cuda.current_device() without its first-call initialisation and
# torch.cuda.current_stream(index).cuda_stream without the Stream object (3 us); a torch
# without CUDA has neither, and its own calls say so
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _stream(stream):
    return _current_stream(_current_device()) if stream is None else stream.cuda_stream


def _may_be_captured(stream):
    """Whether a call on this stream (None: the current one) may have been captured
    into a graph.  torch tells of the current stream only, and raises if it cannot tell
    for another thread's or stream's capture."""
    if not torch.cuda.is_initialized():
        return False
    if stream is not None and stream.cuda_stream != _current_stream(_current_device()):
        return True
    try:
        return torch.cuda.is_current_stream_capturing()
    except RuntimeError:
        return True


class MoELayer:
    """Buffers of one (T, H, E, I, top_k, mode) problem on one device."""

    def __init__(self, T, H, E, I, top_k, mode="bf16", save_for_backward=True,
                 device="cuda", backward=True):
        self.dims = moe_dims(T, H, E, I, top_k, MODES[mode], 1 if save_for_backward else 0)
        self.mode = mode
        self.T, self.H, self.E, self.I, self.k = T, H, E, I, top_k
        self.dtype = torch.float32 if mode == "f32" else torch.bfloat16
        self.device = torch.device(device)
        rows = moe_max_rows(self.dims)
        if rows < 0:
            raise MoEError(1, "invalid dims")
        self.max_rows = rows
        dev = self.device
        i32 = dict(dtype=torch.int32, device=dev)
        self.topk_idx = torch.empty((T, top_k), **i32)
        self.gate = torch.empty((T, top_k), dtype=torch.float32, device=dev)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.padded_offsets = torch.empty(E + 1, **i32)
        self.row_of_assign = torch.empty(T * top_k, **i32)
        self.assign_of_row = torch.empty(rows, **i32)
        self.route_out = moe_route_out(
            _ptr(self.topk_idx), _ptr(self.gate), _ptr(self.counts), _ptr(self.offsets),
            _ptr(self.padded_offsets), _ptr(self.row_of_assign), _ptr(self.assign_of_row))
        u8 = dict(dtype=torch.uint8, device=dev)
        self.ws_route = torch.empty(moe_workspace_size(self.dims, MOE_WS_ROUTE), **u8)
        self.ws_fwd = torch.empty(moe_workspace_size(self.dims, MOE_WS_FORWARD), **u8)
        self.ws_bwd = torch.empty(moe_workspace_size(self.dims, MOE_WS_BACKWARD) if backward else 0,
                                  **u8)
        self.layout = moe_saved_layout_of(self.dims)
        self._saved, self._views = torch.empty(self.layout.total, **u8), {}
        self._no_h13 = None          # where the last forward kept no h13: address and version of `saved`
        self._replays = False        # a forward that keeps h13 has been captured into a graph
        self.status = torch.zeros(4, **i32)

    # ------------------------------------------------------------- views
    @property
    def saved(self):
        """The buffer of saved activations, which may be replaced.  (Whoever takes it may
        also replace its memory, or write it: no view is kept that would hold the old
        one, and what it holds is not known.)"""
        self._views, self._no_h13 = {}, None
        return self._saved

    @saved.setter
    def saved(self, buffer):
        self._views, self._saved, self._no_h13 = {}, buffer, None

    @saved.deleter
    def saved(self):
        self._views = {}
        del self._saved

    def _view(self, offset, rows, cols):
        """Rows of `saved` as it is now, a tensor of its own each time.  (Made from one
        that is kept while the memory stays: 1.1 us instead of 5.8.)"""
        buffer, views = self._saved, self._views
        at = (buffer.data_ptr(), buffer.numel(), self.dtype)
        if views.get("at") != at:
            views = self._views = {"at": at}
        kept = views.get((offset, rows, cols))
        if kept is None:
            n = rows * cols * (4 if self.dtype == torch.float32 else 2)
            kept = buffer[offset:offset + n].view(self.dtype).view(rows, cols)
            if torch.is_inference_mode_enabled():        # (an inference tensor for good)
                return kept
            views[offset, rows, cols] = kept
        return kept.view(rows, cols)

    @property
    def x_perm(self):
        """Gathered tokens [rows, H]; None in mxfp8 mode (not stored)."""
        if self.mode == "mxfp8":
            return None
        return self._view(self.layout.x_perm, self.max_rows, self.H)

    @property
    def act_is_gated(self):
        """bf16 mode stores gate * A in `act` (see moe.h)."""
        return self.mode == "bf16"

    @property
    def h13(self):
        self._no_h13 = None          # (the caller may write it)
        return self._view(self.layout.h13, self.max_rows, 2 * self.I)

    @property
    def act(self):
        """The activation [rows, I] (gate * A in bf16 mode); None in mxfp8
        mode, which keeps A only as its MXFP8 encodings."""
        if self.mode == "mxfp8":
            return None
        return self._view(self.layout.act, self.max_rows, self.I)

    def device_status(self) -> int:
        return int(self.status[0].item())

    def clear_status(self):
        self.status.zero_()

    # ------------------------------------------------------------- calls
    def route(self, logits, stream=None):
        rc = moe_route(self.dims, _ptr(logits), self.route_out, _ptr(self.ws_route),
                       self.ws_route.numel(), _ptr(self.status), _stream(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_route")

    def _route(self, route):
        """The routing of a call: the layer's own, or that of a Router of the same
        tokens, experts and top_k (it has to be on this device)."""
        if route is None:
            return self.route_out
        if (route.T, route.E, route.k) != (self.T, self.E, self.k):
            raise MoEError(MOE_ERR_INVALID_ARG, f"route: expected T, E, top_k = {self.T}, {self.E}, {self.k}; got "
                                                f"{route.T}, {route.E}, {route.k}")
        if route.device != self.gate.device:
            raise MoEError(MOE_ERR_INVALID_ARG, f"route: expected {self.gate.device}; got {route.device}")
        return route.route_out

    def forward(self, X, W13, W2, Y, stream=None, save=None, route=None):
        """save: None = the layer's setting; False = inference, or a first pass
        that is run again before its backward (h13 not kept, so that ``save``
        refuses); True = keep h13 for ``backward`` or ``save``.
        route: a training.Router that holds the routing, in place of the
        layer's own (``route`` above)."""
        dims = self.dims
        if save is not None and bool(save) != bool(self.dims.save_for_backward):
            dims = moe_dims(self.dims.T, self.dims.H, self.dims.E, self.dims.I, self.dims.top_k,
                            self.dims.mode, 1 if save else 0)
        rc = moe_forward(dims, _ptr(X), _ptr(W13), _ptr(W2), self._route(route), _ptr(Y),
                         _ptr(self._saved), self._saved.numel(), _ptr(self.ws_fwd),
                         self.ws_fwd.numel(), _ptr(self.status), _stream(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_forward")
        self._keeps_h13(dims.save_for_backward, stream)

    def _keeps_h13(self, kept, stream):
        """Notes for ``save`` whether `saved` holds this call's h13.  A captured call
        runs when its graph is replayed, which is not seen here; nor are writes to an
        inference tensor."""
        if _may_be_captured(stream):
            self._replays = self._replays or bool(kept)
        else:
            b = self._saved
            self._no_h13 = None if kept or b.is_inference() else (b.data_ptr(), b._version)

    def backward(self, dY, W13, W2, dX, dW13, dW2, dgate, stream=None, route=None):
        rc = moe_backward(self.dims, _ptr(dY), _ptr(W13), _ptr(W2), self._route(route),
                          _ptr(self._saved), self._saved.numel(), _ptr(dX), _ptr(dW13), _ptr(dW2),
                          _ptr(dgate), _ptr(self.ws_bwd), self.ws_bwd.numel(),
                          _ptr(self.status), _stream(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_backward")

    def route_backward(self, dgate, dlogits, stream=None):
        rc = moe_route_backward(self.dims, self.route_out, _ptr(dgate), _ptr(dlogits),
                                _ptr(self.status), _stream(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_route_backward")

    # -------------------------------------------------------- checkpoints
    def checkpoint(self):
        """Buffers that keep one forward's activations in 8 bits (not in mxfp8
        mode)."""
        return Checkpoint(self)

    def _checkpoint(self, checkpoint, X=None):
        if (checkpoint.T, checkpoint.H, checkpoint.I, checkpoint.k) != (self.T, self.H, self.I, self.k):
            raise MoEError(MOE_ERR_INVALID_ARG, "checkpoint: made for a layer of other sizes")
        if checkpoint.device != self.gate.device:
            raise MoEError(MOE_ERR_INVALID_ARG, f"checkpoint: expected {self.gate.device}; got {checkpoint.device}")
        if _current_device() != self.gate.device.index:
            raise MoEError(MOE_ERR_INVALID_ARG, f"called for {self.gate.device}, but another device is current")
        if X is not None and (X.dtype != self.dtype or tuple(X.shape) != (self.T, self.H) or not X.is_contiguous()
                              or X.device != self.gate.device):
            raise MoEError(MOE_ERR_INVALID_ARG, f"X: expected contiguous {self.dtype} [{self.T}, {self.H}] on "
                                                f"{self.gate.device}")
        return checkpoint.pointers

    def save(self, checkpoint, X=None, stream=None, route=None):
        """After ``forward``: X and h13 into the checkpoint, in 8 bits.  X None:
        ``checkpoint.x`` holds its codes already (RMSNorm.forward(encoded=) wrote
        them).  Another forward may then use the layer's buffers.  Refused after a
        forward that kept no h13 (save=False), unless it was written otherwise:
        by ``restore``, by torch, or by whoever looked at ``h13`` or ``saved`` since."""
        none = self._no_h13
        if none and not self._replays and none[0] == self._saved.data_ptr() and none[1] == self._saved._version:
            raise MoEError(MOE_ERR_INVALID_ARG, "save: the last forward kept no h13 (save=False)")
        rc = moe_checkpoint_save(self.dims, None if X is None else _ptr(X), self._route(route), _ptr(self._saved),
                                 self._saved.numel(), self._checkpoint(checkpoint, X), _ptr(self.status),
                                 _stream(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_checkpoint_save")

    def restore(self, checkpoint, stream=None, route=None):
        """Before ``backward``: the saved activations of the checkpoint's
        forward, whose routing ``route`` (or the layer's own) still has to hold."""
        rc = moe_checkpoint_restore(self.dims, self._checkpoint(checkpoint), self._route(route), _ptr(self._saved),
                                    self._saved.numel(), _ptr(self.status), _stream(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_checkpoint_restore")
        self._keeps_h13(True, stream)

    # --------------------------------------------------------- allocation
    def empty_io(self):
        """Output tensors of one forward + backward: Y, dX, dW13, dW2, dgate."""
        dev, dt = self.device, self.dtype
        return dict(
            Y=torch.empty((self.T, self.H), dtype=dt, device=dev),
            dX=torch.empty((self.T, self.H), dtype=dt, device=dev),
            dW13=torch.empty((self.E, self.H, 2 * self.I), dtype=dt, device=dev),
            dW2=torch.empty((self.E, self.I, self.H), dtype=dt, device=dev),
            dgate=torch.empty((self.T, self.k), dtype=torch.float32, device=dev),
        )


class Checkpoint:
    """One forward's activations in 8 bits: the layer's input ``x`` [T, H], and
    ``h13`` [T * top_k, 2I] in the order of the assignments (training.MXRows)."""

    def __init__(self, layer):
        from .training import MXRows
        if layer.mode == "mxfp8":
            raise MoEError(MOE_ERR_UNSUPPORTED, "checkpoint: the mxfp8 mode saves most activations in 8 bits")
        self.T, self.H, self.I, self.k = layer.T, layer.H, layer.I, layer.k
        self.device = layer.gate.device
        self.x, self.h13 = MXRows(self.T, self.H, self.device), MXRows(self.T * self.k, 2 * self.I, self.device)
        self._kept = (self.x, self.h13)          # (whatever becomes of the names)
        self.pointers = moe_checkpoint(_ptr(self.x.codes), _ptr(self.x.scales), _ptr(self.h13.codes),
                                       _ptr(self.h13.scales))
