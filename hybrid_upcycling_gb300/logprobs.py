"""Log-probabilities of given tokens, with entropy and top alternatives, as PyTorch functions.

``token_logprobs(logits, tokens)`` takes logits; ``head_logprobs(h, W, tokens)`` takes final hidden states
and the LM head and never stores the logits. Log-probabilities and entropies of both are
differentiable. They run in the sm_103a kernels of libhylo_kl.so through the C ABI
(include/hylo_ops.h); PyTorch only allocates the outputs and the workspace.
"""
from __future__ import annotations

from typing import NamedTuple, Tuple

import torch

from . import _lib


class TokenLogprobs(NamedTuple):
    logprobs: torch.Tensor      # [...]: log-probability of each given token (0 where it is negative)
    entropy: torch.Tensor       # [...]: entropy of each distribution, in nats
    top_logprobs: torch.Tensor  # [..., top_k], largest first
    top_tokens: torch.Tensor    # [..., top_k] int64; equal logits: lowest token first


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
        return torch.empty(N, V, dtype=z.dtype, device=z.device)
    buf = torch.empty(lead + N * ld, dtype=z.dtype, device=z.device)
    return buf.as_strided((N, V), (ld, 1), lead)


def _forward(z, tokens, tau, k, train):
    N = z.shape[0]
    f = dict(dtype=torch.float32, device=z.device)
    logp, entropy = torch.empty(N, **f), torch.empty(N, **f)
    stats = torch.empty(N, 2, **f) if train else None
    top = torch.empty(N, k, **f)
    ids = torch.empty(N, k, dtype=torch.int64, device=z.device)
    if N > 0:
        _lib.hylo_token_logprobs(z, tokens, tau, k, logp, entropy, None, stats, top, ids)
    return logp, entropy, top, ids, stats


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, z, tokens, tau, k):
        logp, entropy, top, ids, stats = _forward(z, tokens, tau, k, True)
        ctx.save_for_backward(z, tokens, stats, entropy)
        ctx.tau = tau
        ctx.mark_non_differentiable(top, ids)
        ctx.set_materialize_grads(False)
        return logp, entropy, top, ids

    @staticmethod
    def backward(ctx, g_logp, g_entropy, _top, _ids):
        z, tokens, stats, entropy = ctx.saved_tensors
        dz = _grad_rows(z)
        if z.shape[0] > 0:
            g_logp, g_entropy = (None if g is None else g.float().contiguous() for g in (g_logp, g_entropy))
            _lib.hylo_token_logprobs_backward(z, tokens, ctx.tau, stats, entropy, g_logp, g_entropy, dz)
        return dz, None, None, None


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, tau: float = 1.0, top_k: int = 0) -> TokenLogprobs:
    """Log-probabilities of ``tokens`` [...] (int64) under softmax(logits / tau), logits [..., V] in float32,
    bfloat16 or float16, with each distribution's entropy and its ``top_k`` (<= 64) most probable tokens.

    logits may have any strides; rows with unit column stride are read in place. A negative token is
    ignored (log-probability 0, no gradient); -inf logits are masked words. logprobs and entropy
    are differentiable with respect to logits (gradient in the logits' dtype)."""
    if logits.dtype not in _lib.DTYPES or logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError("logits must be float32, bfloat16 or float16 with a last dimension of at least one word")
    if tokens.dtype != torch.int64 or tokens.shape != logits.shape[:-1]:
        raise ValueError("tokens must be int64 with the shape of logits without its last dimension")
    if not 0 <= top_k <= min(_lib.TOP_MAX, logits.shape[-1]):
        raise ValueError(f"top_k must be in [0, min(V, {_lib.TOP_MAX})]")
    z, t = _rows(logits), tokens.reshape(-1).contiguous()
    if torch.is_grad_enabled() and logits.requires_grad:
        r = _TokenLogprobs.apply(z, t, float(tau), int(top_k))
    else:
        r = _forward(z, t, float(tau), int(top_k), False)
    logp, entropy, top, ids = r[:4]
    if tokens.dim() != 1:
        logp, entropy = logp.view(tokens.shape), entropy.view(tokens.shape)
        top, ids = top.view(*tokens.shape, top_k), ids.view(*tokens.shape, top_k)
    return TokenLogprobs(logp, entropy, top, ids)


def _workspace(h, W, token_chunk, split_g):
    N, d = h.shape
    n = _lib.hylo_head_logprobs_workspace_bytes(N, d, W.shape[0], token_chunk, split_g)
    if n == 0:
        raise ValueError("invalid sizes (the hidden size must be a multiple of 8 in 8..65536)")
    return torch.empty(n, dtype=torch.uint8, device=h.device)  # from the caching allocator of the current stream


def _head_forward(h, W, tokens, tau, train):
    N = h.shape[0]
    f = dict(dtype=torch.float32, device=h.device)
    logp, entropy = torch.empty(N, **f), torch.empty(N, **f)
    lse = torch.empty(N, **f) if train else None
    if N > 0:
        _lib.hylo_head_logprobs(h, W, tokens, tau, logp, entropy, lse, _workspace(h, W, 0, False))
    return logp, entropy, lse


class _HeadLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, W, tokens, tau, token_chunk, split_g):
        logp, entropy, lse = _head_forward(h, W, tokens, tau, True)
        ctx.save_for_backward(h, W, tokens, lse, entropy)
        ctx.args = (tau, token_chunk, split_g)
        ctx.set_materialize_grads(False)
        return logp, entropy

    @staticmethod
    def backward(ctx, g_logp, g_entropy):
        h, W, tokens, lse, entropy = ctx.saved_tensors
        tau, token_chunk, split_g = ctx.args
        if h.shape[0] == 0:
            return torch.zeros_like(h), torch.zeros_like(W), None, None, None, None
        f = dict(dtype=torch.float32, device=h.device)
        dh, dW = torch.empty(h.shape, **f), torch.empty(W.shape, **f)
        g_logp, g_entropy = (None if g is None else g.float().contiguous() for g in (g_logp, g_entropy))
        _lib.hylo_head_logprobs_backward(h, W, tokens, tau, token_chunk, lse, entropy, g_logp, g_entropy, dh, dW,
                                         _workspace(h, W, token_chunk, split_g), split_g)
        return (dh.to(h.dtype) if ctx.needs_input_grad[0] else None, dW.to(W.dtype) if ctx.needs_input_grad[1] else None,
                None, None, None, None)


def head_logprobs(h: torch.Tensor, W: torch.Tensor, tokens: torch.Tensor, tau: float = 1.0, token_chunk: int = 4096,
                  split_g: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Log-probabilities of ``tokens`` [...] (int64) under softmax(h W^T / tau) and the entropies, for final hidden
    states h [..., d] and an LM head W [V, d] in bfloat16 (d a multiple of 8); the logits are never stored.

    A negative token is ignored (log-probability 0, no gradient). Both results are differentiable
    with respect to h and W (bfloat16 gradients; the C ABI gives fp32). token_chunk and split_g as in
    fused_hidden_state_kl: the backward's token block, and whether the gradient of the logits is
    kept to 16 bits of precision instead of 8 inside the gradient products."""
    if h.dtype != torch.bfloat16 or W.dtype != torch.bfloat16 or h.dim() < 1 or W.dim() != 2 or h.shape[-1] != W.shape[1]:
        raise ValueError("h [..., d] and W [V, d] must be bfloat16 with the same hidden size")
    if tokens.dtype != torch.int64 or tokens.shape != h.shape[:-1]:
        raise ValueError("tokens must be int64 with the shape of h without its last dimension")
    hh, WW, t = h.reshape(-1, h.shape[-1]).contiguous(), W.contiguous(), tokens.reshape(-1).contiguous()
    if torch.is_grad_enabled() and (h.requires_grad or W.requires_grad):
        logp, entropy = _HeadLogprobs.apply(hh, WW, t, float(tau), int(token_chunk), bool(split_g))
    else:
        logp, entropy, _ = _head_forward(hh, WW, t, float(tau), False)
    return logp.view(tokens.shape), entropy.view(tokens.shape)
