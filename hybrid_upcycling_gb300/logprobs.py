"""Log-probabilities of given tokens, with entropy and top alternatives, as PyTorch functions.

``token_logprobs(logits, tokens)`` takes logits; its log-probabilities and entropies are
differentiable. It runs in the sm_103a kernels of libhylo_kl.so through the C ABI
(include/hylo_ops.h); PyTorch only allocates the outputs.
"""
from __future__ import annotations

from typing import NamedTuple

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
