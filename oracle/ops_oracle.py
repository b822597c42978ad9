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


# ------------------------------------------------------------------------------------------------ norms
def norm(s, weight, bias, eps: float, rms: bool):
    """(y, mean [N, 1], 1 / deviation [N, 1]) of rows s [N, d]; weight and bias [d] or None."""
    s = np.asarray(s, np.float64)
    mu = np.zeros((s.shape[0], 1)) if rms else s.mean(axis=1, keepdims=True)
    r = 1 / np.sqrt(((s - mu) ** 2).mean(axis=1, keepdims=True) + eps)
    y = (s - mu) * r
    if weight is not None:
        y = y * weight
    return (y if bias is None else y + bias), mu, r


def norm_grad(s, weight, eps: float, rms: bool, dy):
    """Gradients (ds, dweight, dbias) of sum(dy y), from the derivatives of mean and deviation one by one."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    _, mu, r = norm(s, None, None, eps, rms)
    c, d = s - mu, s.shape[1]
    g = dy if weight is None else dy * weight
    dr = (g * c).sum(axis=1, keepdims=True)             # y = c r
    dvar = -0.5 * r ** 3 * dr                           # r = (var + eps)^(-1/2)
    dc = g * r + dvar * 2 * c / d                       # var = mean(c^2)
    ds = dc if rms else dc - dc.mean(axis=1, keepdims=True)
    return ds, (dy * c * r).sum(axis=0), dy.sum(axis=0)


# ------------------------------------------------------------------------------- orthogonalised updates
MUON = (3.4445, -4.7750, 2.0315)


def orthogonalize(x, coefficients=(MUON,) * 5, eps: float = 1e-7) -> np.ndarray:
    """Newton-Schulz steps from x / (|x| + eps), one (a, b, c) a step; a matrix of zeros gives zeros."""
    x = np.asarray(x, np.float64)
    norm = np.sqrt((x ** 2).sum())
    if norm == 0:
        return np.zeros_like(x)
    x = x / (norm + eps)
    if x.shape[0] > x.shape[1]:
        return _steps(x.T, coefficients).T
    return _steps(x, coefficients)


def _steps(x, coefficients):
    for a, b, c in coefficients:
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def orthogonalize_fp16(x, coefficients=(MUON,) * 5, eps: float = 1e-7) -> np.ndarray:
    """The same with the roundings of the fp16 scheme: X as two fp16 terms, the products with the first; A and
    B = b A + c A^2 in fp16, all scaled far from fp16's limits; sums exact."""
    def half(v):  # fp16 of v 2^14 (entries are at most about 3)
        return (v * 2.0 ** 14).astype(np.float16).astype(np.float64) / 2.0 ** 14

    x = np.asarray(x, np.float64)
    norm = np.sqrt((x ** 2).sum())
    if norm == 0:
        return np.zeros_like(x)
    x = x / (norm + eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    for a, b, c in coefficients:
        hi = half(x)
        lo = half(x - hi)
        g = half(hi @ hi.T)
        x = a * (hi + lo) + half(b * g + c * (g @ g)) @ hi
    x = half(x)
    return x.T if tall else x


def muon(w, g, m, *, lr, momentum, nesterov, weight_decay, scale, coefficients=(MUON,) * 5, eps=1e-7):
    """One step in fp64: (w, m)."""
    w, g, m = (np.asarray(t, np.float64) for t in (w, g, m))
    m = momentum * m + (1 - momentum) * g
    u = momentum * m + (1 - momentum) * g if nesterov else m
    return w * (1 - lr * weight_decay) - lr * scale * orthogonalize(u, coefficients, eps), m
