"""Caller-side buffers of the operators around the expert layer in a training
step: layer norm, cross entropy over a vocabulary, and gradient clipping.

As in ``layer``, PyTorch supplies device memory and the stream; every
computation is a call into libmoe_gb300.so.  Each class owns the statistics
and the workspace of one problem shape on one device, checks the tensors it is
given against that shape, and raises ``MoEError`` on any non-OK return code, for
tensors that do not fit and while another device is current.

An object's calls on different streams, or from different threads, have to be
ordered by the caller, since they share its buffers (a LayerNorm with
``backward=False`` has none to share); and it has to live until work that it put
on a stream other than the one it was made on is done.
"""
from __future__ import annotations

import torch

from . import (MOE_ERR_INVALID_ARG, MOE_INDEX_I32, MOE_INDEX_I64, MOE_OK, MOE_REDUCE_MEAN,
               MOE_REDUCE_NONE, MOE_REDUCE_SUM, MOE_TYPE_BF16, MOE_TYPE_F32, MOE_WS_BACKWARD,
               MOE_WS_FORWARD, MoEError, moe_clip_grads, moe_cross_entropy,
               moe_cross_entropy_backward, moe_cross_entropy_workspace_size, moe_grad_norm,
               moe_grad_tensor, moe_grad_workspace_size, moe_layer_norm, moe_layer_norm_backward,
               moe_layer_norm_workspace_size, moe_norm_dims, moe_xent_dims)
from .layer import _ptr

TYPES = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}
INDEX_TYPES = {torch.int32: MOE_INDEX_I32, torch.int64: MOE_INDEX_I64}
REDUCTIONS = {"none": MOE_REDUCE_NONE, "sum": MOE_REDUCE_SUM, "mean": MOE_REDUCE_MEAN}


# torch.cuda.current_stream(index).cuda_stream without the Stream object (3 us),
# torch.cuda.current_device() without its first-call initialisation
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _require(ok, what):
    if not ok:
        raise MoEError(MOE_ERR_INVALID_ARG, what)


def _require_int32(what, *numbers):
    # (ctypes would keep the low 32 bits of others)
    _require(all(-(1 << 31) <= n < 1 << 31 for n in numbers), what + ": sizes and ignored values have 32 bits")


class _Op:
    """The checks cost about as much as a small kernel, so they are a few
    comparisons each and build no text unless something is wrong."""

    def _fits(self, name, t, shape, dtype):
        """`t` is a contiguous tensor of this shape and type on this device;
        returns its address."""
        try:
            ok = (t.dtype is dtype and t.shape == shape and t.get_device() == self.index
                  and t.is_contiguous())
        except AttributeError:
            ok = False
        if not ok:
            self._refuse(name, t, shape, dtype, "contiguous")
        return t.data_ptr()

    def _fits_or_none(self, name, t, shape, dtype):
        return None if t is None else self._fits(name, t, shape, dtype)

    def _rows(self, name, t, shape, dtype):
        """As _fits, for rows of adjacent elements that may lie apart (a slice
        of a wider buffer); returns the address and the distance of rows."""
        try:
            ok = t.dtype is dtype and t.shape == shape and t.get_device() == self.index
            ld, step = t.stride()
        except (AttributeError, ValueError):
            ok = False
        rows, cols = shape
        if ok and rows <= 1:
            ld = cols
        if not ok or ld < cols or (step != 1 and cols > 1 and rows > 0):
            self._refuse(name, t, shape, dtype, "adjacent elements in rows that do not overlap")
        return t.data_ptr(), ld

    @property
    def dims(self):
        """The library's description of the problem, as of the last call."""
        return self._described[1]

    def _keep(self, *tensors):
        """Keeps the memory of tensors whose addresses are recorded."""
        self._kept = tensors

    def _refuse(self, name, t, shape, dtype, layout):
        got = f"{t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}" \
            if isinstance(t, torch.Tensor) else repr(t)
        raise MoEError(MOE_ERR_INVALID_ARG, f"{name}: expected {dtype} {tuple(shape)} on {self.device}, "
                                            f"{layout}; got {got}")

    def _current(self, stream):
        """Handle of `stream`, or of the device's current stream.  The library
        launches on the thread's current device, so that has to be this one."""
        if _current_device() != self.index or (
                stream is not None and getattr(stream, "device_index", self.index) != self.index):
            raise MoEError(MOE_ERR_INVALID_ARG, f"called for {self.device}, but cuda:{_current_device()} "
                                                f"is current (stream: {stream})")
        return _current_stream(self.index) if stream is None else stream.cuda_stream

    def _device(self, device):
        d = torch.device(device)
        self.index = torch.cuda.current_device() if d.index is None else d.index
        self.device = torch.device("cuda", self.index)

    def device_status(self) -> int:
        return int(self.status[0].item())

    def clear_status(self):
        self.status.zero_()


class LayerNorm(_Op):
    """Layer norm of [T, H] rows, float32 or bfloat16, with weights of either
    type.  x, y, dy and dx may be slices of wider buffers."""

    def __init__(self, T, H, dtype=torch.bfloat16, weight_dtype=None, eps=1e-5, device="cuda",
                 backward=True):
        weight_dtype = dtype if weight_dtype is None else weight_dtype
        _require(dtype in TYPES and weight_dtype in TYPES, "LayerNorm: float32 or bfloat16")
        _require_int32("LayerNorm", T, H)
        self.T, self.H, self.dtype, self.weight_dtype, self.eps = T, H, dtype, weight_dtype, eps
        self._device(device)
        self.shape = torch.Size((T, H))
        self._described = (None, None)
        need = moe_layer_norm_workspace_size(self._dims(H, H, H))
        _require(need > 0, "LayerNorm: invalid sizes")
        f32 = dict(dtype=torch.float32, device=self.device)
        self.mean = torch.empty(T, **f32) if backward else None
        self.rstd = torch.empty(T, **f32) if backward else None
        self._keep(self.mean, self.rstd)
        self._stats = (_ptr(self.mean), _ptr(self.rstd))
        self.ws = torch.empty(need if backward else 0, dtype=torch.uint8, device=self.device)

    def _dims(self, *lds):
        """The library's description with these distances of rows.  A published
        one is never written again: a call in another thread may be reading it."""
        known = self._described
        if known[0] != lds:
            known = self._described = (lds, moe_norm_dims(self.T, self.H, *lds, TYPES[self.dtype],
                                                          TYPES[self.weight_dtype], self.eps))
        return known[1]

    def forward(self, x, gamma, beta, y, stream=None):
        """y = layer norm of x; gamma and beta may be None (1 and 0)."""
        shape, dt, wt, w = self.shape, self.dtype, self.weight_dtype, self.shape[1:]
        x, ld_x = self._rows("x", x, shape, dt)
        y, ld_y = self._rows("y", y, shape, dt)
        gamma = self._fits_or_none("gamma", gamma, w, wt)
        beta = self._fits_or_none("beta", beta, w, wt)
        rc = moe_layer_norm(self._dims(ld_x, ld_y, self.H), x, gamma, beta, y, *self._stats,
                            self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_layer_norm")

    def backward(self, dy, x, gamma, dx, dgamma=None, dbeta=None, stream=None):
        """dx, dgamma and dbeta (None leaves one out) of the last forward's x."""
        shape, dt, wt, w = self.shape, self.dtype, self.weight_dtype, self.shape[1:]
        _require(self.mean is not None, "LayerNorm: built with backward=False")
        dy, ld_dy = self._rows("dy", dy, shape, dt)
        x, ld_x = self._rows("x", x, shape, dt)
        dx, ld_dx = self._rows("dx", dx, shape, dt)
        gamma = self._fits_or_none("gamma", gamma, w, wt)
        dgamma = self._fits_or_none("dgamma", dgamma, w, wt)
        dbeta = self._fits_or_none("dbeta", dbeta, w, wt)
        rc = moe_layer_norm_backward(self._dims(ld_x, ld_dy, ld_dx), dy, x, gamma, *self._stats, dx, dgamma,
                                     dbeta, self.ws.data_ptr(), self.ws.numel(), self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_layer_norm_backward")

    def empty_io(self):
        """Output tensors: y, dx, dgamma, dbeta."""
        x = dict(dtype=self.dtype, device=self.device)
        w = dict(dtype=self.weight_dtype, device=self.device)
        return dict(y=torch.empty((self.T, self.H), **x), dx=torch.empty((self.T, self.H), **x),
                    dgamma=torch.empty(self.H, **w), dbeta=torch.empty(self.H, **w))


class CrossEntropy(_Op):
    """Softmax cross entropy of bfloat16 hidden states X [T, H] against the
    output weights W [V, H], logits not kept.  After ``forward``: ``loss`` and
    ``lse`` [T], and ``sum``, ``mean`` and ``count`` over the rows that count
    (all float32 on the device)."""

    def __init__(self, T, H, V, ignore_index=-100, index_dtype=torch.int64, device="cuda",
                 backward=True):
        _require(index_dtype in INDEX_TYPES, "CrossEntropy: int32 or int64 targets")
        _require_int32("CrossEntropy", T, H, V, ignore_index)
        self.T, self.H, self.V, self.ignore_index = T, H, V, ignore_index
        self.index_dtype = index_dtype
        self._device(device)
        self._described = (None, None)
        dims = self._dims(H, H)
        need = moe_cross_entropy_workspace_size(dims, MOE_WS_FORWARD)
        _require(need > 0, "CrossEntropy: invalid sizes (H has to be a multiple of 8)")
        if backward:
            # the two calls of a step run one after the other: one workspace
            need = max(need, moe_cross_entropy_workspace_size(dims, MOE_WS_BACKWARD))
        f32 = dict(dtype=torch.float32, device=self.device)
        self.loss = torch.empty(T, **f32)
        self.lse = torch.empty(T, **f32)
        self.total = torch.empty(3, **f32)
        self.sum, self.mean, self.count = self.total[0], self.total[1], self.total[2]
        self.ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self.with_backward = backward
        self._keep(self.loss, self.lse, self.total)
        self._out = (self.loss.data_ptr(), self.lse.data_ptr(), self.total.data_ptr())

    def _dims(self, *lds):
        """As LayerNorm's."""
        known = self._described
        if known[0] != lds:
            known = self._described = (lds, moe_xent_dims(self.T, self.H, self.V, *lds, self.ignore_index,
                                                          INDEX_TYPES[self.index_dtype]))
        return known[1]

    def _inputs(self, X, W, targets):
        X, ld_x = self._rows("X", X, (self.T, self.H), torch.bfloat16)
        W, ld_w = self._rows("W", W, (self.V, self.H), torch.bfloat16)
        return self._dims(ld_x, ld_w), X, W, self._fits("targets", targets, (self.T,), self.index_dtype)

    def forward(self, X, W, targets, stream=None):
        d, X, W, targets = self._inputs(X, W, targets)
        rc = moe_cross_entropy(d, X, W, targets, *self._out, self.ws.data_ptr(), self.ws.numel(),
                               self.status.data_ptr(), self._current(stream))
        if rc != MOE_OK:
            self._failed(rc, "moe_cross_entropy", d, X=X, W=W)

    def backward(self, X, W, targets, dloss, dX, dW, reduction="mean", stream=None):
        """dX and dW (None leaves one out) after ``forward`` on the same inputs.
        dloss: the gradient of each row's loss [T] (reduction "none"), or of
        their sum or mean, [] or [1]."""
        _require(self.with_backward, "CrossEntropy: built with backward=False")
        _require(reduction in REDUCTIONS, "CrossEntropy: reduction is none, sum or mean")
        d, X, W, targets = self._inputs(X, W, targets)
        shape = (self.T,) if reduction == "none" else () if getattr(dloss, "ndim", 1) == 0 else (1,)
        dloss = self._fits("dloss", dloss, shape, torch.float32)
        dX = self._fits_or_none("dX", dX, (self.T, self.H), torch.bfloat16)
        dW = self._fits_or_none("dW", dW, (self.V, self.H), torch.bfloat16)
        _, lse, total = self._out
        rc = moe_cross_entropy_backward(d, X, W, targets, lse, total, dloss, REDUCTIONS[reduction], dX,
                                        dW, self.ws.data_ptr(), self.ws.numel(),
                                        self.status.data_ptr(), self._current(stream))
        if rc != MOE_OK:
            self._failed(rc, "moe_cross_entropy_backward", d, X=X, W=W, dX=dX, dW=dW)

    def _failed(self, rc, call, d, **addresses):
        """Names the tensors whose rows do not all start on 16-byte boundaries."""
        ld = dict(X=d.ld_x, W=d.ld_w)
        off = [k for k, p in addresses.items() if p and p % 16 or ld.get(k, 0) % 8]
        raise MoEError(rc, f"{call}: {', '.join(off)}: rows have to start on 16-byte boundaries" if off else call)

    def empty_io(self):
        """Output tensors of the backward: dX, dW."""
        b = dict(dtype=torch.bfloat16, device=self.device)
        return dict(dX=torch.empty((self.T, self.H), **b), dW=torch.empty((self.V, self.H), **b))


_address = torch.Tensor.data_ptr


class GradClip(_Op):
    """Global L2 norm of a list of gradient tensors (contiguous, float32 or
    bfloat16), and clipping by it: in place, or into the tensors `out`.  Where
    the tensors lie is looked up at every call (their ``data`` may have been
    replaced since); a size that changes in the same place is not noticed, and
    the memory given before stays in use.  After either call ``norm`` [] holds
    the norm (float32 on the device)."""

    def __init__(self, grads, out=None, device="cuda"):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        _require(len(self.out) == len(self.grads), "GradClip: as many outputs as gradients")
        self._device(self.grads[0].device if self.grads else device)
        self._tensors = self.grads if out is None else self.grads + self.out
        self._describe()
        self.norm = torch.empty((), dtype=torch.float32, device=self.device)
        self.ws = torch.empty(moe_grad_workspace_size(len(self.grads)), dtype=torch.uint8,
                              device=self.device)
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self._keep(self.norm, self.ws, self.status)
        self._buffers = (self.norm.data_ptr(), self.ws.data_ptr(), self.ws.numel(),
                         self.status.data_ptr())

    def _describe(self):
        """Checks the tensors and lists them for the library."""
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            _require(isinstance(g, torch.Tensor) and g.dtype in TYPES, f"grads[{i}]: float32 or bfloat16")
            self._fits(f"grads[{i}]", g, g.shape, g.dtype)
            self._fits(f"out[{i}]", o, g.shape, g.dtype)
        entries = (moe_grad_tensor * max(1, len(self.grads)))(
            *[moe_grad_tensor(_ptr(g), _ptr(o), g.numel(), TYPES[g.dtype])
              for g, o in zip(self.grads, self.out)])
        # (aliases of their own, which keep the listed memory whatever becomes of the tensors)
        self._listed = (entries, list(map(_address, self._tensors)), [t.detach() for t in self._tensors])
        return entries

    def _list(self):
        """The list, made again if a tensor lies elsewhere.  (0.08 us per tensor;
        without it a freed address would be written to.  Sizes too: twice that.)"""
        entries, addresses, _ = self._listed
        return entries if list(map(_address, self._tensors)) == addresses else self._describe()

    def measure(self, stream=None):
        """The norm alone."""
        rc = moe_grad_norm(self._list(), len(self.grads), *self._buffers, self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_grad_norm")

    def clip(self, max_norm, stream=None):
        """out = grads * min(1, max_norm / norm)."""
        rc = moe_clip_grads(self._list(), len(self.grads), max_norm, *self._buffers, self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_clip_grads")
