"""Caller-side buffers of the operators around the expert layer in a training
step: layer norm, cross entropy over a vocabulary, and gradient clipping.

As in ``layer``, PyTorch supplies device memory and the stream; every
computation is a call into libmoe_gb300.so.  Each class owns the statistics
and the workspace of one problem shape on one device, checks the tensors it
is given against that shape, and raises ``MoEError`` on any non-OK return code
and for tensors that do not fit.
"""
from __future__ import annotations

import torch

from . import (MOE_ERR_INVALID_ARG, MOE_INDEX_I32, MOE_INDEX_I64, MOE_OK, MOE_REDUCE_MEAN,
               MOE_REDUCE_NONE, MOE_REDUCE_SUM, MOE_TYPE_BF16, MOE_TYPE_F32, MOE_WS_BACKWARD,
               MOE_WS_FORWARD, MoEError, moe_clip_grads, moe_cross_entropy,
               moe_cross_entropy_backward, moe_cross_entropy_workspace_size, moe_grad_norm,
               moe_grad_tensor, moe_grad_workspace_size, moe_layer_norm, moe_layer_norm_backward,
               moe_layer_norm_workspace_size, moe_norm_dims, moe_xent_dims)
from .layer import _ptr, _stream

TYPES = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16}
INDEX_TYPES = {torch.int32: MOE_INDEX_I32, torch.int64: MOE_INDEX_I64}
REDUCTIONS = {"none": MOE_REDUCE_NONE, "sum": MOE_REDUCE_SUM, "mean": MOE_REDUCE_MEAN}


def _require(ok, what):
    if not ok:
        raise MoEError(MOE_ERR_INVALID_ARG, what)


def _call(rc, what):
    if rc != MOE_OK:
        raise MoEError(rc, what)


class _Op:
    def _fits(self, name, t, shape, dtype, strided=False, optional=False):
        """`t` has this shape and type on this device, contiguous or (strided)
        with rows of adjacent elements."""
        if t is None and optional:
            return
        _require(isinstance(t, torch.Tensor) and t.dtype == dtype and tuple(t.shape) == tuple(shape)
                 and t.device == self.device, f"{name}: expected {dtype} {tuple(shape)} on {self.device}")
        if strided:
            _require(t.numel() == 0 or t.shape[1] == 1 or t.stride(1) == 1,
                     f"{name}: rows of adjacent elements are expected")
            _require(self._ld(t) >= t.shape[1], f"{name}: overlapping rows")
        else:
            _require(t.is_contiguous(), f"{name}: a contiguous tensor is expected")

    @staticmethod
    def _ld(t):
        """Elements from one row of `t` to the next."""
        return t.stride(0) if t.shape[0] > 1 else t.shape[1]

    def _device(self, device):
        d = torch.device(device)
        self.device = torch.device("cuda", torch.cuda.current_device()) if d.index is None else d

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
        self.T, self.H, self.dtype, self.weight_dtype, self.eps = T, H, dtype, weight_dtype, eps
        self._device(device)
        need = moe_layer_norm_workspace_size(self._dims(H, H, H))
        _require(need > 0, "LayerNorm: invalid sizes")
        f32 = dict(dtype=torch.float32, device=self.device)
        self.mean = torch.empty(T, **f32) if backward else None
        self.rstd = torch.empty(T, **f32) if backward else None
        self.ws = torch.empty(need if backward else 0, dtype=torch.uint8, device=self.device)

    def _dims(self, ld_x, ld_y, ld_dx):
        return moe_norm_dims(self.T, self.H, ld_x, ld_y, ld_dx, TYPES[self.dtype],
                             TYPES[self.weight_dtype], self.eps)

    def forward(self, x, gamma, beta, y, stream=None):
        """y = layer norm of x; gamma and beta may be None (1 and 0)."""
        T, H = self.T, self.H
        for n, t in (("x", x), ("y", y)):
            self._fits(n, t, (T, H), self.dtype, strided=True)
        for n, t in (("gamma", gamma), ("beta", beta)):
            self._fits(n, t, (H,), self.weight_dtype, optional=True)
        _call(moe_layer_norm(self._dims(self._ld(x), self._ld(y), H), _ptr(x), _ptr(gamma), _ptr(beta),
                             _ptr(y), _ptr(self.mean), _ptr(self.rstd), _stream(stream)),
              "moe_layer_norm")

    def backward(self, dy, x, gamma, dx, dgamma=None, dbeta=None, stream=None):
        """dx, dgamma and dbeta (None leaves one out) of the last forward's x."""
        T, H = self.T, self.H
        _require(self.mean is not None, "LayerNorm: built with backward=False")
        for n, t in (("dy", dy), ("x", x), ("dx", dx)):
            self._fits(n, t, (T, H), self.dtype, strided=True)
        for n, t in (("gamma", gamma), ("dgamma", dgamma), ("dbeta", dbeta)):
            self._fits(n, t, (H,), self.weight_dtype, optional=True)
        _call(moe_layer_norm_backward(self._dims(self._ld(x), self._ld(dy), self._ld(dx)), _ptr(dy),
                                      _ptr(x), _ptr(gamma), _ptr(self.mean), _ptr(self.rstd), _ptr(dx),
                                      _ptr(dgamma), _ptr(dbeta), _ptr(self.ws), self.ws.numel(),
                                      _stream(stream)), "moe_layer_norm_backward")

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
        self.T, self.H, self.V, self.ignore_index = T, H, V, ignore_index
        self.index_dtype = index_dtype
        self._device(device)
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

    def _dims(self, ld_x, ld_w):
        return moe_xent_dims(self.T, self.H, self.V, ld_x, ld_w, self.ignore_index,
                             INDEX_TYPES[self.index_dtype])

    def _inputs(self, X, W, targets):
        self._fits("X", X, (self.T, self.H), torch.bfloat16, strided=True)
        self._fits("W", W, (self.V, self.H), torch.bfloat16, strided=True)
        self._fits("targets", targets, (self.T,), self.index_dtype)
        return self._dims(self._ld(X), self._ld(W))

    def forward(self, X, W, targets, stream=None):
        dims = self._inputs(X, W, targets)
        _call(moe_cross_entropy(dims, _ptr(X), _ptr(W), _ptr(targets), _ptr(self.loss), _ptr(self.lse),
                                _ptr(self.total), _ptr(self.ws), self.ws.numel(), _ptr(self.status),
                                _stream(stream)), "moe_cross_entropy")

    def backward(self, X, W, targets, dloss, dX, dW, reduction="mean", stream=None):
        """dX and dW (None leaves one out) after ``forward`` on the same inputs.
        dloss: the gradient of each row's loss [T] (reduction "none"), or of
        their sum or mean [1]."""
        dims = self._inputs(X, W, targets)
        _require(self.with_backward, "CrossEntropy: built with backward=False")
        _require(reduction in REDUCTIONS, "CrossEntropy: reduction is none, sum or mean")
        self._fits("dloss", dloss, (self.T if reduction == "none" else 1,), torch.float32)
        self._fits("dX", dX, (self.T, self.H), torch.bfloat16, optional=True)
        self._fits("dW", dW, (self.V, self.H), torch.bfloat16, optional=True)
        _call(moe_cross_entropy_backward(dims, _ptr(X), _ptr(W), _ptr(targets), _ptr(self.lse),
                                         _ptr(self.total), _ptr(dloss), REDUCTIONS[reduction], _ptr(dX),
                                         _ptr(dW), _ptr(self.ws), self.ws.numel(), _ptr(self.status),
                                         _stream(stream)), "moe_cross_entropy_backward")

    def empty_io(self):
        """Output tensors of the backward: dX, dW."""
        b = dict(dtype=torch.bfloat16, device=self.device)
        return dict(dX=torch.empty((self.T, self.H), **b), dW=torch.empty((self.V, self.H), **b))


class GradClip(_Op):
    """Global L2 norm of a fixed list of gradient tensors (contiguous, float32
    or bfloat16), and clipping by it: in place, or into the tensors `out`.
    After either call ``norm`` [] holds the norm (float32 on the device)."""

    def __init__(self, grads, out=None, device="cuda"):
        self.grads = list(grads)
        self.out = self.grads if out is None else list(out)
        _require(len(self.out) == len(self.grads), "GradClip: as many outputs as gradients")
        self._device(self.grads[0].device if self.grads else device)
        for i, (g, o) in enumerate(zip(self.grads, self.out)):
            _require(isinstance(g, torch.Tensor) and g.dtype in TYPES, f"grads[{i}]: float32 or bfloat16")
            self._fits(f"grads[{i}]", g, g.shape, g.dtype)
            self._fits(f"out[{i}]", o, g.shape, g.dtype)
        self.list = (moe_grad_tensor * max(1, len(self.grads)))(
            *[moe_grad_tensor(_ptr(g), _ptr(o), g.numel(), TYPES[g.dtype])
              for g, o in zip(self.grads, self.out)])
        self.norm = torch.empty((), dtype=torch.float32, device=self.device)
        self.ws = torch.empty(moe_grad_workspace_size(len(self.grads)), dtype=torch.uint8,
                              device=self.device)
        self.status = torch.zeros(4, dtype=torch.int32, device=self.device)

    def measure(self, stream=None):
        """The norm alone."""
        _call(moe_grad_norm(self.list, len(self.grads), _ptr(self.norm), _ptr(self.ws),
                            self.ws.numel(), _ptr(self.status), _stream(stream)), "moe_grad_norm")

    def clip(self, max_norm, stream=None):
        """out = grads * min(1, max_norm / norm)."""
        _call(moe_clip_grads(self.list, len(self.grads), max_norm, _ptr(self.norm), _ptr(self.ws),
                             self.ws.numel(), _ptr(self.status), _stream(stream)), "moe_clip_grads")
