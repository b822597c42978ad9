"""Layer norm and RMS norm over the last dimension, with the sum of the residual stream in the same pass.

``layer_norm(x, weight, bias)`` and ``rms_norm(x, weight)`` are differentiable PyTorch functions that run in the sm_103a
kernels of libhylo_kl.so through the C ABI (include/hylo_ops.h has the formulas); PyTorch only allocates the
outputs and the workspace.
"""
from __future__ import annotations

from typing import Optional, Tuple, Union

import torch
from torch.autograd.forward_ad import unpack_dual

from . import _lib
from ._lib import _check, _ptr, current_raw_stream, load
from .logprobs import _on_device, _row_stride, _rows

_empty, _f32 = torch.empty, torch.float32


def _forward(x, residual, weight, bias, gain, eps, rms, dev, train):
    N, d = x.shape
    device = x.device
    y = _empty((N, d), dtype=x.dtype, device=device)
    total = None if residual is None else _empty((N, d), dtype=x.dtype, device=device)
    stats = _empty((N, 2), dtype=_f32, device=device) if train else None
    if N > 0:
        _check(load().hylo_norm(
            x.data_ptr(), _ptr(residual), _lib.DTYPES[x.dtype], N, d, _row_stride(x),
            0 if residual is None else _row_stride(residual), _ptr(weight), _ptr(bias), gain, rms, eps, _ptr(total),
            y.data_ptr(), _ptr(stats), current_raw_stream(dev)))
    return y, total, stats


class _Once(torch.autograd.Function):
    """A gradient, as a function of `inputs` whose own derivative is not implemented."""
    @staticmethod
    def forward(ctx, grad, *inputs):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("layer_norm and rms_norm are differentiable once")


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, bias, gain, eps, rms, dev):
        y, total, stats = _forward(x, residual, weight, bias, gain, eps, rms, dev, True)
        ctx.save_for_backward(x if total is None else total, weight, stats)
        ctx.args = (gain, rms, None if bias is None else bias.dtype)
        ctx.set_materialize_grads(False)
        return y if total is None else (y, total)

    @staticmethod
    def backward(ctx, dy, dsum=None):
        s, weight, stats = ctx.saved_tensors
        gain, rms, bias_dtype = ctx.args
        want_x, want_r, want_w, want_b = ctx.needs_input_grad[:4]
        N, d = s.shape
        device = s.device
        dx = dw = db = None
        if dy is None or N == 0:  # nothing comes through the norm
            if want_x or want_r:
                dx = dsum if dsum is not None else None if dy is None else torch.zeros_like(dy)
            dw = torch.zeros_like(weight) if want_w else None
            db = torch.zeros(d, dtype=bias_dtype, device=device) if want_b else None
        else:
            dy, dsum = _rows(dy), None if dsum is None else _rows(dsum)
            if want_x or want_r:
                dx = _empty((N, d), dtype=s.dtype, device=device)
            if want_w:
                dw = _empty(d, dtype=weight.dtype, device=device)
            if want_b:
                db = _empty(d, dtype=bias_dtype, device=device)
            ws, n = None, 0
            if want_w or want_b:
                n = load().hylo_norm_backward_workspace_bytes(N, d)
                ws = _empty(n, dtype=torch.uint8, device=device)  # from the caching allocator of the current stream
            _check(load().hylo_norm_backward(
                s.data_ptr(), _lib.DTYPES[s.dtype], N, d, _row_stride(s), _ptr(weight), gain, rms, stats.data_ptr(),
                dy.data_ptr(), _row_stride(dy), _ptr(dsum), 0 if dsum is None else _row_stride(dsum), _ptr(dx), _ptr(dw),
                _ptr(db), _ptr(ws), n, current_raw_stream(s.get_device())))
        if torch.is_grad_enabled():  # create_graph
            inputs = [t for t in (s, weight, dy, dsum) if t is not None]
            dx, dw, db = (None if g is None else _Once.apply(g, *inputs) for g in (dx, dw, db))
        return dx if want_x else None, dx if want_r else None, dw, db, None, None, None, None


def _norm(x, weight, bias, eps, residual, rms):
    shape = x.shape
    if x.dtype not in _lib.DTYPES or not shape or shape[-1] < 1:
        raise ValueError("x must be float32, bfloat16 or float16 with a last dimension of at least one element")
    d = shape[-1]
    if residual is not None and (residual.dtype != x.dtype or residual.shape != shape):
        raise ValueError("residual must have the dtype and shape of x")
    gain, tensors = x.dtype, [x]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is None:
            continue
        if t.shape != (d,) or t.dtype not in (x.dtype, _f32):
            raise ValueError(f"{name} must be [{d}], float32 or of the dtype of x")
        if len(tensors) > 1 and t.dtype != gain:
            raise ValueError("weight and bias must have the same dtype")
        gain = t.dtype
        tensors.append(t)
    if residual is not None:
        tensors.append(residual)
    for t in tensors:
        if unpack_dual(t).tangent is not None:
            raise NotImplementedError("layer_norm and rms_norm have no forward-mode derivatives")
    dev = _on_device(*tensors)
    rows, r = _rows(x), None if residual is None else _rows(residual)
    w, b = None if weight is None else weight.contiguous(), None if bias is None else bias.contiguous()
    if torch.is_grad_enabled() and any(t.requires_grad for t in tensors):
        out = _Norm.apply(rows, r, w, b, _lib.DTYPES[gain], float(eps), int(rms), dev)
        y, total = out if residual is not None else (out, None)
    else:
        y, total, _ = _forward(rows, r, w, b, _lib.DTYPES[gain], float(eps), int(rms), dev, False)
    if len(shape) != 2:
        y, total = y.view(shape), None if total is None else total.view(shape)
    return y if residual is None else (y, total)


Normed = Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]


def layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
               eps: float = 1e-5, residual: Optional[torch.Tensor] = None) -> Normed:
    """Layer norm of x [..., d] (float32, bfloat16 or float16) over its last dimension: (x - mean) / sqrt(variance + eps)
    times ``weight`` [d] plus ``bias`` [d] (either may be left out; both of x's dtype or both float32).

    With ``residual`` (shape and dtype of x) the norm is that of the sum, and (norm, sum) is returned, the sum rounded to
    x's dtype as the next layer reads it. x may have any strides; rows with unit column stride are read in place.
    Differentiable once, in reverse mode, with respect to every tensor; only the gradients that are needed are computed."""
    return _norm(x, weight, bias, eps, residual, False)


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None) -> Normed:
    """RMS norm of x [..., d]: x / sqrt(mean(x^2) + eps) times ``weight`` [d]. Everything else as in ``layer_norm``."""
    return _norm(x, weight, None, eps, residual, True)
