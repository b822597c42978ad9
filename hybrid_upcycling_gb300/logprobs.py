"""Log-probabilities of given tokens, with entropy and top alternatives, as PyTorch functions.

``token_logprobs(logits, tokens)`` takes logits; ``head_logprobs(h, W, tokens)`` takes final hidden states
and the LM head and never stores the logits. Log-probabilities and entropies of both are
differentiable. They run in the sm_103a kernels of libhylo_kl.so through the C ABI
(include/hylo_ops.h); PyTorch only allocates the outputs and the workspace.

A decoding loop calls these once per token, so each tensor is looked at once and the C entry points are
called directly (the functions of the same names in ``_lib`` check their arguments a second time).
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch
from torch.autograd.forward_ad import unpack_dual

from . import _lib
from ._lib import _check, current_raw_stream, load

_empty, _f32 = torch.empty, torch.float32
_BF16 = _lib.DTYPES[torch.bfloat16]


class TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor      # [...]: log-probability of each given token (0 where it is negative)
    entropy: torch.Tensor       # [...]: entropy of each distribution, in nats
    top_logprobs: torch.Tensor  # [..., top_k], largest first
    top_tokens: torch.Tensor    # [..., top_k] int64; equal logits: lowest token first


def _on_device(*tensors: torch.Tensor) -> int:
    """The current CUDA device, which must be that of every tensor."""
    if not tensors[0].is_cuda:
        raise ValueError("the tensors must be CUDA tensors")
    dev = torch.cuda.current_device()
    for t in tensors:
        if t.get_device() != dev:
            raise ValueError(f"every tensor must be on the current CUDA device ({dev})")
    return dev


def _no_tangents(*tensors: torch.Tensor) -> None:
    for t in tensors:
        if unpack_dual(t).tangent is not None:
            raise NotImplementedError("token_logprobs and head_logprobs have no forward-mode derivatives")


def _row_stride(z: torch.Tensor) -> int:
    return z.stride(0) if z.shape[0] > 1 else max(z.shape[1], z.stride(0))


def _rows(z: torch.Tensor) -> torch.Tensor:
    """z [..., V] as [N, V] rows with unit column stride that do not overlap: a view where it can be one."""
    V = z.shape[-1]
    z = z.reshape(-1, V) if z.dim() != 2 else z
    if (V > 1 and z.stride(1) != 1) or (z.shape[0] > 1 and z.stride(0) < V):
        z = z.contiguous()
    return z


def _grad_rows(z: torch.Tensor) -> torch.Tensor:
    """An uninitialised [N, V] gradient whose rows lie at z's rows' offsets modulo 16 bytes (so that both are
    read and written in the same 16-byte vectors)."""
    N, V = z.shape
    unit = 16 // z.element_size()
    lead = z.data_ptr() % 16 // z.element_size()
    ld = V + (z.stride(0) - V) % unit if N > 1 else V
    if lead == 0 and ld == V:
        return _empty((N, V), dtype=z.dtype, device=z.device)
    buf = _empty(lead + N * ld, dtype=z.dtype, device=z.device)
    return buf.as_strided((N, V), (ld, 1), lead)


def _forward(z, tokens, tau, k, dev, train):
    N, V = z.shape
    device = z.device
    logp, entropy = _empty(N, dtype=_f32, device=device), _empty(N, dtype=_f32, device=device)
    stats = _empty((N, 2), dtype=_f32, device=device) if train else None
    top, ids = _empty((N, k), dtype=_f32, device=device), _empty((N, k), dtype=torch.int64, device=device)
    if N > 0:
        _check(load().hylo_token_logprobs(
            z.data_ptr(), _lib.DTYPES[z.dtype], N, V, _row_stride(z), tau, tokens.data_ptr(), k, logp.data_ptr(),
            entropy.data_ptr(), None, stats.data_ptr() if train else None, top.data_ptr(), ids.data_ptr(),
            current_raw_stream(dev)))
    return logp, entropy, top, ids, stats


def _upstream(g):
    return g if g is None or (g.dtype is _f32 and g.is_contiguous()) else g.to(_f32).contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


class _Once(torch.autograd.Function):
    """A gradient, as a function of `inputs` whose own derivative is not implemented."""
    @staticmethod
    def forward(ctx, grad, *inputs):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("token_logprobs and head_logprobs are differentiable once")


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, tokens, tau, k, dev, alternatives):
        logp, entropy, top, ids, stats = _forward(z, tokens, tau, k, dev, True)
        alternatives += (top, ids)  # not differentiable
        ctx.save_for_backward(z, tokens, stats, entropy)
        ctx.tau = tau
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    def backward(ctx, g_logp, g_entropy):
        z, tokens, stats, entropy = ctx.saved_tensors
        dz = _grad_rows(z)
        N, V = z.shape
        if N > 0:
            g_logp, g_entropy = _upstream(g_logp), _upstream(g_entropy)
            _check(load().hylo_token_logprobs_backward(
                z.data_ptr(), _lib.DTYPES[z.dtype], N, V, _row_stride(z), ctx.tau, tokens.data_ptr(), stats.data_ptr(),
                entropy.data_ptr(), _ptr(g_logp), _ptr(g_entropy), dz.data_ptr(), _row_stride(dz),
                current_raw_stream(z.get_device())))
        if torch.is_grad_enabled():  # create_graph
            dz = _Once.apply(dz, z, g_logp, g_entropy)
        return dz, None, None, None, None, None


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, tau: float = 1.0, top_k: int = 0) -> TokenLogprobs:
    """Log-probabilities of ``tokens`` [...] (int64) under softmax(logits / tau), logits [..., V] in float32,
    bfloat16 or float16, with each distribution's entropy and its ``top_k`` (<= 64) most probable tokens.

    logits may have any strides; rows with unit column stride are read in place. A negative token is
    ignored (log-probability 0, no gradient); -inf logits are masked words. logprobs and entropy
    are differentiable once, in reverse mode, with respect to logits (gradient in the logits' dtype)."""
    shape = logits.shape
    if logits.dtype not in _lib.DTYPES or not shape or shape[-1] < 1:
        raise ValueError("logits must be float32, bfloat16 or float16 with a last dimension of at least one word")
    if tokens.dtype != torch.int64 or tokens.shape != shape[:-1]:
        raise ValueError("tokens must be int64 with the shape of logits without its last dimension")
    if not 0 <= top_k <= min(_lib.TOP_MAX, shape[-1]):
        raise ValueError(f"top_k must be in [0, min(V, {_lib.TOP_MAX})]")
    _no_tangents(logits)
    dev = _on_device(logits, tokens)
    plain = len(shape) == 2
    z, t = _rows(logits), (tokens if plain else tokens.reshape(-1)).contiguous()
    if logits.requires_grad and torch.is_grad_enabled():
        alternatives = []
        logp, entropy = _TokenLogprobs.apply(z, t, float(tau), int(top_k), dev, alternatives)
        top, ids = alternatives
    else:
        logp, entropy, top, ids, _ = _forward(z, t, float(tau), int(top_k), dev, False)
    if not plain:
        logp, entropy = logp.view(tokens.shape), entropy.view(tokens.shape)
        top, ids = top.view(*tokens.shape, top_k), ids.view(*tokens.shape, top_k)
    return TokenLogprobs(logp, entropy, top, ids)


def _workspace(n, device):
    if n == 0:
        raise ValueError("invalid sizes (the hidden size must be a multiple of 8 in 8..65536)")
    return _empty(n, dtype=torch.uint8, device=device), n  # from the caching allocator of the current stream


def _head_forward(h, W, tokens, tau, dev, train):
    (N, d), V = h.shape, W.shape[0]
    device = h.device
    logp, entropy = _empty(N, dtype=_f32, device=device), _empty(N, dtype=_f32, device=device)
    lse = _empty(N, dtype=_f32, device=device) if train else None
    if N > 0:
        ws, n = _workspace(load().hylo_head_logprobs_forward_workspace_bytes(N, d, V), device)
        _check(load().hylo_head_logprobs(h.data_ptr(), W.data_ptr(), N, d, V, tau, tokens.data_ptr(), logp.data_ptr(),
                                         entropy.data_ptr(), _ptr(lse), ws.data_ptr(), n, current_raw_stream(dev)))
    return logp, entropy, lse


class _HeadLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, tokens, tau, token_chunk, split_g, dev):
        logp, entropy, lse = _head_forward(h, W, tokens, tau, dev, True)
        ctx.save_for_backward(h, W, tokens, lse, entropy)
        ctx.args = (tau, token_chunk, split_g)
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    def backward(ctx, g_logp, g_entropy):
        h, W, tokens, lse, entropy = ctx.saved_tensors
        tau, token_chunk, split_g = ctx.args
        (N, d), V = h.shape, W.shape[0]
        want_h, want_W = ctx.needs_input_grad[:2]
        if N == 0:
            return (torch.zeros_like(h) if want_h else None, torch.zeros_like(W) if want_W else None, None, None, None, None,
                    None)
        dh, dW = torch.empty_like(h) if want_h else None, torch.empty_like(W) if want_W else None
        g_logp, g_entropy = _upstream(g_logp), _upstream(g_entropy)
        ws, n = _workspace(load().hylo_head_logprobs_backward_workspace_bytes(
            N, d, V, token_chunk, int(split_g), _BF16, int(want_h), int(want_W)), h.device)
        _check(load().hylo_head_logprobs_backward(
            h.data_ptr(), W.data_ptr(), N, d, V, tau, token_chunk, tokens.data_ptr(), lse.data_ptr(), entropy.data_ptr(),
            _ptr(g_logp), _ptr(g_entropy), int(split_g), _BF16, _ptr(dh), _ptr(dW), ws.data_ptr(), n,
            current_raw_stream(h.get_device())))
        if torch.is_grad_enabled():  # create_graph
            dh, dW = (None if g is None else _Once.apply(g, h, W, g_logp, g_entropy) for g in (dh, dW))
        return dh, dW, None, None, None, None, None


def head_logprobs(h: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor, tau: float = 1.0, token_chunk: int = 4096,
                  split_g: Optional[bool] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Log-probabilities of ``tokens`` [...] (int64) under softmax(h W^T / tau) and the entropies, for final hidden
    states h [..., d] and an LM head W [V, d] in bfloat16 (d a multiple of 8); the logits are never stored.

    A negative token is ignored (log-probability 0, no gradient). Both results are differentiable once, in
    reverse mode, with respect to h and W (bfloat16 gradients; the C ABI gives fp32), and only the gradients
    that are needed are computed. token_chunk and split_g as in fused_hidden_state_kl: the backward's token
    block, and whether the gradient of the logits is kept to 16 bits of precision instead of 8 inside the gradient
    products (None: for up to 64 tokens, where that rounding does not average out: relative error 3e-3 of the
    gradients against 1.7e-3 with both terms)."""
    shape = h.shape
    if h.dtype != torch.bfloat16 or W.dtype != torch.bfloat16 or not shape or W.dim() != 2 or shape[-1] != W.shape[1]:
        raise ValueError("h [..., d] and W [V, d] must be bfloat16 with the same hidden size")
    if tokens.dtype != torch.int64 or tokens.shape != shape[:-1]:
        raise ValueError("tokens must be int64 with the shape of h without its last dimension")
    _no_tangents(h, W)
    dev = _on_device(h, W, tokens)
    plain = len(shape) == 2
    hh, t = (h, tokens) if plain else (h.reshape(-1, shape[-1]), tokens.reshape(-1))
    hh, WW, t = hh.contiguous(), W.contiguous(), t.contiguous()
    if (h.requires_grad or W.requires_grad) and torch.is_grad_enabled():
        logp, entropy = _HeadLogprobs.apply(hh, WW, t, float(tau), int(token_chunk),
                                            hh.shape[0] <= 64 if split_g is None else bool(split_g), dev)
    else:
        logp, entropy, _ = _head_forward(hh, WW, t, float(tau), dev, False)
    return (logp, entropy) if plain else (logp.view(tokens.shape), entropy.view(tokens.shape))
