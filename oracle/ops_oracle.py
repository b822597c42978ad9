"""fp64 CPU oracle of the token log-probabilities and of the AdamW step.

TEST INFRASTRUCTURE ONLY, like kl_oracle: it shares no code with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def log_probs(z: np.ndarray, tau: float) -> np.ndarray:
    """log softmax(z / tau) by rows of fp64 logits; -inf logits have probability 0; a row of only -inf gives -inf."""
    y = np.asarray(z, np.float64) / tau
    m = y.max(axis=1, keepdims=True)
    y = y - np.where(np.isneginf(m), 0.0, m)
    with np.errstate(divide="ignore"):
        s = np.exp(y).sum(axis=1, keepdims=True)
        return np.where(s > 0, y - np.log(np.where(s > 0, s, 1.0)), -np.inf)


def token_logprobs(z, tokens, tau: float = 1.0, k: int = 0):
    """(logp [N], entropy [N], top_logp [N, k], top_ids [N, k]) from the definition; ties to the lowest index."""
    z = np.asarray(z, np.float64)
    lp = log_probs(z, tau)
    n = np.arange(z.shape[0])
    t = np.asarray(tokens)
    logp = np.where(t < 0, 0.0, lp[n, np.maximum(t, 0)])
    fin = np.where(np.isneginf(lp), 0.0, lp)
    entropy = -(np.exp(lp) * fin).sum(axis=1)
    ids = np.argsort(-(z + 0.0), axis=1, kind="stable")[:, :k]
    return logp, entropy, np.take_along_axis(lp, ids, 1), ids


def token_logprobs_grad(z, tokens, tau: float, g_logp, g_entropy) -> np.ndarray:
    """d(sum g_logp logp + g_entropy entropy) / dz, element by element from the definition."""
    z = np.asarray(z, np.float64)
    lp = log_probs(z, tau)
    p = np.exp(lp)
    fin = np.where(np.isneginf(lp), 0.0, lp)
    H = -(p * fin).sum(axis=1, keepdims=True)
    t = np.asarray(tokens)
    gl = np.where(t < 0, 0.0, np.asarray(g_logp, np.float64))[:, None]
    one = np.zeros_like(p)
    one[np.arange(len(t)), np.maximum(t, 0)] = 1.0
    d = (gl * (one - p) - np.asarray(g_entropy, np.float64)[:, None] * p * (fin + H)) / tau
    return np.where(np.isneginf(lp).all(axis=1, keepdims=True), 0.0, d)


# ------------------------------------------------------------------------------------------------ AdamW
def mix32(x):
    """The 32-bit finaliser of MurmurHash3 on uint64 arrays that hold 32-bit values."""
    m = np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x85EBCA6B)) & m
    x = ((x ^ (x >> np.uint64(13))) * np.uint64(0xC2B2AE35)) & m
    return x ^ (x >> np.uint64(16))


def random_bits(seed: int, start: int, n: int) -> np.ndarray:
    """32 random bits for positions start .. start + n - 1 of the list of tensors (as uint64)."""
    c = np.arange(start, start + n, dtype=np.uint64)
    m = np.uint64(0xFFFFFFFF)
    key = mix32((np.uint64(seed & 0xFFFFFFFF) + np.uint64(0x9E3779B9) * (((c >> np.uint64(32)) + np.uint64(1)) & m)) & m)
    return mix32(((c & m) + key) & m)


def code_parts(x, block: int = 256):
    """Per element: the step of the e4m3 grid at |x| 2^-e, and |x| 2^-e / step; per block: e."""
    n = len(x)
    a = np.abs(np.pad(np.asarray(x, np.float64), (0, -n % block))).reshape(-1, block)
    top = a.max(axis=1)
    with np.errstate(divide="ignore"):
        e = np.clip(np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 7, -120), -120, 120)
    y = (a * np.exp2(-e)[:, None]).reshape(-1)[:n]
    step = np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    return y / step, step, e


def round_code(x, bits16, keep: bool):
    """(codes as values, exponents): stochastic rounding with 16 random bits; keep: a non-zero is not stored as 0."""
    r, step, e = code_parts(x)
    q = np.floor(r + bits16.astype(np.float64) / 65536) * step
    if keep:
        q = np.where((r > 0) & (q == 0), 2.0 ** -9, q)
    return q * np.sign(x), e


def adamw(w, g, m, v, *, step, lr, betas, eps, weight_decay, clip: float = 1.0):
    """(w, m, v) after one step, fp64."""
    b1, b2 = betas
    g = np.asarray(g, np.float64) * clip
    m = b1 * np.asarray(m, np.float64) + (1 - b1) * g
    v = b2 * np.asarray(v, np.float64) + (1 - b2) * g * g
    w = np.asarray(w, np.float64) * (1 - lr * weight_decay)
    w = w - lr * (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return w, m, v
