"""Caller-side buffers of the operators around the expert layer in a training
step: routing by scores, layer norm, RMS norm, rows in MXFP8, cross entropy over
a vocabulary, and gradient clipping.

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
               MOE_REDUCE_NONE, MOE_REDUCE_SUM, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, MOE_TYPE_BF16,
               MOE_TYPE_F32, MOE_WS_BACKWARD, MOE_WS_FORWARD, MoEError, moe_balance_bias, moe_clip_grads,
               moe_cross_entropy, moe_cross_entropy_backward, moe_cross_entropy_workspace_size,
               moe_dequantize_mxfp8, moe_grad_norm, moe_grad_tensor, moe_grad_workspace_size,
               moe_layer_norm, moe_layer_norm_backward, moe_layer_norm_workspace_size, moe_norm_dims,
               moe_quantize_mxfp8, moe_rms_dims, moe_rms_norm, moe_rms_norm_backward,
               moe_rms_norm_workspace_size, moe_route_out, moe_router, moe_router_backward,
               moe_router_dims, moe_router_workspace_size, moe_xent_dims)
from .layer import _current_device, _current_stream, _ptr

TYPES = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}
INDEX_TYPES = {torch.int32: MOE_INDEX_I32, torch.int64: MOE_INDEX_I64}
SCORES = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
REDUCTIONS = {"none": MOE_REDUCE_NONE, "sum": MOE_REDUCE_SUM, "mean": MOE_REDUCE_MEAN}


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


class RMSNorm(_Op):
    """RMS norm of [T, H] rows with the residual's addition, float32 or bfloat16,
    with weights of either type.  All row tensors may be slices of wider buffers."""

    def __init__(self, T, H, dtype=torch.bfloat16, weight_dtype=None, eps=1e-6, device="cuda", backward=True):
        weight_dtype = dtype if weight_dtype is None else weight_dtype
        _require(dtype in TYPES and weight_dtype in TYPES, "RMSNorm: float32 or bfloat16")
        _require_int32("RMSNorm", T, H)
        self.T, self.H, self.dtype, self.weight_dtype, self.eps = T, H, dtype, weight_dtype, eps
        self._device(device)
        self.shape = torch.Size((T, H))
        self._described = (None, None)
        need = moe_rms_norm_workspace_size(self._dims(H, H, H, H, H, H))
        _require(need > 0, "RMSNorm: invalid sizes")
        self.rstd = torch.empty(T, dtype=torch.float32, device=self.device) if backward else None
        self.ws = torch.empty(need if backward else 0, dtype=torch.uint8, device=self.device)
        self._keep(self.rstd, self.ws)
        self._rstd, self._ws, self._width = _ptr(self.rstd), (self.ws.data_ptr(), self.ws.numel()), self.shape[1:]

    def _dims(self, *lds):
        """As LayerNorm's."""
        known = self._described
        if known[0] != lds:
            known = self._described = (lds, moe_rms_dims(self.T, self.H, *lds, TYPES[self.dtype],
                                                         TYPES[self.weight_dtype], self.eps))
        return known[1]

    def forward(self, x, gamma, y=None, residual=None, h=None, encoded=None, stream=None):
        """h = x + residual, y = h / rms(h) * gamma; gamma may be None (1).  Of h
        (only with a residual), y and encoded (an MXRows: y in 8 bits) those that
        are given are written."""
        shape, dt, H = self.shape, self.dtype, self.H
        if residual is None and h is not None:
            _require(False, "RMSNorm: h is x itself without a residual")
        x, ld_x = self._rows("x", x, shape, dt)
        residual, ld_r = (None, H) if residual is None else self._rows("residual", residual, shape, dt)
        h, ld_h = (None, H) if h is None else self._rows("h", h, shape, dt)
        y, ld_y = (None, H) if y is None else self._rows("y", y, shape, dt)
        if gamma is not None:
            gamma = self._fits("gamma", gamma, self._width, self.weight_dtype)
        q, scales = (None, None) if encoded is None else encoded._pointers("encoded", self)
        rc = moe_rms_norm(self._dims(ld_x, ld_r, ld_h, ld_y, H, H), x, residual, gamma, h, y, q, scales,
                          self._rstd, self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_rms_norm")

    def backward(self, dy, h, gamma, dx, dgamma=None, dh=None, stream=None):
        """dx (of x and of residual) and dgamma (None leaves it out) of the last
        forward, whose sum is h; dh: the gradient that reaches h on other ways."""
        _require(self.rstd is not None, "RMSNorm: built with backward=False")
        shape, dt, H = self.shape, self.dtype, self.H
        dy, ld_dy = self._rows("dy", dy, shape, dt)
        h, ld_h = self._rows("h", h, shape, dt)
        dh, ld_dh = (None, H) if dh is None else self._rows("dh", dh, shape, dt)
        dx, ld_dx = self._rows("dx", dx, shape, dt)
        if gamma is not None:
            gamma = self._fits("gamma", gamma, self._width, self.weight_dtype)
        if dgamma is not None:
            dgamma = self._fits("dgamma", dgamma, self._width, self.weight_dtype)
        rc = moe_rms_norm_backward(self._dims(H, H, ld_h, ld_dy, ld_dh, ld_dx), dy, h, dh, gamma, self._rstd, dx,
                                   dgamma, *self._ws, self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_rms_norm_backward")

    def empty_io(self):
        """Output tensors: y, h, dx, dgamma."""
        x = dict(dtype=self.dtype, device=self.device)
        return dict(y=torch.empty((self.T, self.H), **x), h=torch.empty((self.T, self.H), **x),
                    dx=torch.empty((self.T, self.H), **x),
                    dgamma=torch.empty(self.H, dtype=self.weight_dtype, device=self.device))


class MXRows(_Op):
    """[rows, cols] numbers as MXFP8: ``codes`` (E4M3, uint8) and a scale per 32
    columns, ``scales`` (E8M0, uint8)."""

    def __init__(self, rows, cols, device="cuda"):
        _require_int32("MXRows", rows, cols)
        _require(rows >= 0 and cols >= 0 and cols % 32 == 0, "MXRows: columns in blocks of 32")
        self.rows, self.cols = rows, cols
        self._device(device)
        u8 = dict(dtype=torch.uint8, device=self.device)
        self.codes, self.scales = torch.empty((rows, cols), **u8), torch.empty((rows, cols // 32), **u8)
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)
        self._keep(self.codes, self.scales, self.status)
        self._at, self._shape = (_ptr(self.codes), _ptr(self.scales)), torch.Size((rows, cols))

    def _pointers(self, name, op):
        """The addresses, for an operator whose rows they are to be."""
        if self.rows != op.T or self.cols != op.H or self.index != op.index:
            raise MoEError(MOE_ERR_INVALID_ARG, f"{name}: expected [{op.T}, {op.H}] on {op.device}; got "
                                                f"[{self.rows}, {self.cols}] on {self.device}")
        return self._at

    def encode(self, x, stream=None):
        """From bfloat16 rows that start on 16-byte boundaries."""
        x, ld = self._rows("x", x, self._shape, torch.bfloat16)
        _require(ld < 1 << 31, "MXRows: rows less than 2^31 elements apart")
        rc = moe_quantize_mxfp8(x, self.rows, self.cols, ld, 1, None, 0, *self._at, self.status.data_ptr(),
                                self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_quantize_mxfp8")

    def decode(self, out, stream=None):
        """The values into bfloat16 or float32 rows."""
        dtype = getattr(out, "dtype", None)
        kind = TYPES.get(dtype)
        if kind is None:
            _require(False, "MXRows: float32 or bfloat16")
        out, ld = self._rows("out", out, self._shape, dtype)
        rc = moe_dequantize_mxfp8(*self._at, self.rows, self.cols, ld, kind, out, self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_dequantize_mxfp8")


class Router(_Op):
    """Routing of T tokens to top_k of E experts by softmax or sigmoid scores,
    with a bias for balance, groups of experts, and gates that are renormalised
    or not, times ``scale``.  After ``forward`` the arrays of moe_route_out
    (``topk_idx``, ``gate``, ``counts``, ...) hold the routing, which
    ``MoELayer.forward`` and ``backward`` take as ``route``."""

    def __init__(self, T, E, top_k, score="softmax", groups=1, top_groups=1, group_top=1, renormalise=True,
                 scale=1.0, dtype=torch.float32, device="cuda"):
        _require(dtype in TYPES, "Router: float32 or bfloat16 logits")
        _require(score in SCORES, "Router: softmax or sigmoid")
        _require_int32("Router", T, E, top_k, groups, top_groups, group_top)
        self.T, self.E, self.k, self.dtype = T, E, top_k, dtype
        self._how = (TYPES[dtype], SCORES[score], groups, top_groups, group_top, 1 if renormalise else 0, scale)
        self._device(device)
        self._described = (None, None)
        need = moe_router_workspace_size(self._dims(E))
        _require(need > 0, "Router: invalid sizes")
        i32 = dict(dtype=torch.int32, device=self.device)
        self.topk_idx = torch.empty((T, top_k), **i32)
        self.gate = torch.empty((T, top_k), dtype=torch.float32, device=self.device)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.padded_offsets = torch.empty(E + 1, **i32)
        self.row_of_assign = torch.empty(T * top_k, **i32)
        self.assign_of_row = torch.empty(T * top_k + 128 * E, **i32)
        self.ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        self.status = torch.zeros(4, **i32)
        arrays = (self.topk_idx, self.gate, self.counts, self.offsets, self.padded_offsets, self.row_of_assign,
                  self.assign_of_row)
        self._keep(*arrays, self.ws, self.status)
        self.route_out = moe_route_out(*map(_ptr, arrays))
        self._shape, self._counts, self._status = torch.Size((T, E)), self.counts.data_ptr(), self.status.data_ptr()
        self._experts, self._chosen = torch.Size((E,)), torch.Size((T, top_k))
        self._ws = (self.ws.data_ptr(), need)

    def _dims(self, ld):
        """As LayerNorm's."""
        known = self._described
        if known[0] != ld:
            known = self._described = (ld, moe_router_dims(self.T, self.E, self.k, ld, *self._how))
        return known[1]

    def forward(self, logits, bias=None, stream=None):
        """logits [T, E] (a slice of a wider buffer too); bias [E] float32 or None."""
        logits, ld = self._rows("logits", logits, self._shape, self.dtype)
        if bias is not None:
            bias = self._fits("bias", bias, self._experts, torch.float32)
        rc = moe_router(self._dims(ld), logits, bias, self.route_out, *self._ws, self._status,
                        self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_router")

    def backward(self, logits, dgate, dlogits, stream=None):
        """dlogits [T, E] of the last forward's logits, from dgate [T, top_k]."""
        logits, ld = self._rows("logits", logits, self._shape, self.dtype)
        dgate = self._fits("dgate", dgate, self._chosen, torch.float32)
        dlogits = self._fits("dlogits", dlogits, self._shape, self.dtype)
        rc = moe_router_backward(self._dims(ld), self.route_out, logits, dgate, dlogits, self._status,
                                 self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_router_backward")

    def update_bias(self, bias, rate, out=None, stream=None):
        """Moves the bias by ``rate`` towards an even load, by the last forward's
        counts: in place, or into ``out``."""
        bias = self._fits("bias", bias, self._experts, torch.float32)
        out = bias if out is None else self._fits("out", out, self._experts, torch.float32)
        rc = moe_balance_bias(self.E, self._counts, rate, bias, out, self._current(stream))
        if rc != MOE_OK:
            raise MoEError(rc, "moe_balance_bias")


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
