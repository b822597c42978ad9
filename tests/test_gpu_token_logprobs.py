"""GPU parity of token_logprobs (forward, alternatives, gradient) against the fp64 oracle.

Tolerances, with u = 2^-24. A thread adds at most n = V / 256 + 32 positive terms in fp32 before tree sums, so log s
is off by at most (n + 16) u and, through the rounded exponents y (|y| e^y <= 1 on average a few units), a few
u more: logp and top_logp within (n + 64) u (1 + |x|), entropy (a quotient of two such sums) within
twice that. A gradient element d = p (A + B log p) is off by its rounding to the logits' type and by
(n + 128) 2u of the magnitudes that make it up.
"""
import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, head_logprobs, token_logprobs
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_ULP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # 2^-p, p significant bits
TINY = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}  # half the step of subnormals
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def f64(t):
    return t.detach().double().cpu().numpy()


def logits(N, V, dtype, seed=0, std=1.3, pad=0, shift=0):
    """[N, V] logits in rows of V + pad, the first row `shift` elements off a 16-byte boundary."""
    gen = torch.Generator("cuda").manual_seed(seed)
    buf = torch.full((N * (V + pad) + shift,), 60.0, dtype=dtype, device="cuda")
    z = buf[shift:].view(N, V + pad)[:, :V]
    z.copy_(torch.randn(N, V, generator=gen, device="cuda") * std)
    tok = torch.randint(0, V, (N,), generator=gen, device="cuda")
    return z, tok


def near(x, ref, tol):
    x = f64(x)
    assert np.array_equal(np.isnan(x), np.isnan(ref))
    inf = np.isinf(ref)
    assert np.array_equal(x[inf], ref[inf])
    ok = ~inf & ~np.isnan(ref)
    err = np.abs(x[ok] - ref[ok]) / (1 + np.abs(ref[ok]))
    assert err.size == 0 or err.max() <= tol, err.max()


def check(z, tok, tau=1.0, k=8, grad=True, seed=1):
    N, V = z.shape
    z = z.detach().requires_grad_(grad)
    r = token_logprobs(z, tok, tau=tau, top_k=k)
    zz, tt = f64(z), tok.cpu().numpy()
    lp, H, top, ids = oo.token_logprobs(zz, tt, tau, k)
    n = V / 256 + 32
    near(r.logprobs, lp, (n + 64) * U)
    near(r.entropy, H, 2 * (n + 64) * U)
    near(r.top_logprobs, top, (n + 64) * U)
    assert np.array_equal(r.top_tokens.cpu().numpy(), ids)
    if grad:
        rng = np.random.default_rng(seed)
        gl, ge = rng.normal(size=N), rng.normal(size=N)
        gl, ge = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (gl, ge))
        for a, b in ((gl, ge), (gl, None), (None, ge)):
            outs = [(o, g) for o, g in ((r.logprobs, a), (r.entropy, b)) if g is not None]
            dz, = torch.autograd.grad([o for o, _ in outs], [z], [g for _, g in outs], retain_graph=True)
            A, B = (np.zeros(N) if g is None else f64(g) for g in (a, b))
            ref = oo.token_logprobs_grad(zz, tt, tau, A, B)
            llp = oo.log_probs(zz, tau)
            p, fin = np.exp(llp), np.where(np.isneginf(llp), 0.0, llp)
            size = p * (np.abs(A)[:, None] + np.abs(B)[:, None] * (np.abs(fin) + H[:, None])) / tau
            size[np.arange(N), np.maximum(tt, 0)] += np.abs(A) / tau
            tol = HALF_ULP[z.dtype] * np.abs(ref) * 1.01 + TINY[z.dtype] + (n + 128) * 2 * U * size + 1e-38
            assert dz.dtype == z.dtype and dz.shape == z.shape
            bad = np.abs(f64(dz) - ref) > tol
            assert not bad.any(), (np.argwhere(bad)[:3], np.abs(f64(dz) - ref)[bad][:3], tol[bad][:3])
    return r


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,pad,shift,tau,k", [
    (1, 1, 0, 0, 1.0, 1), (3, 2, 0, 1, 0.5, 2), (5, 7, 3, 0, 2.0, 3), (2, 255, 0, 3, 1.0, 64), (3, 256, 0, 0, 1.0, 20),
    (4, 257, 5, 1, 1.0, 64), (7, 1000, 0, 5, 0.7, 1), (5, 4096, 8, 0, 1.0, 16), (3, 33001, 0, 7, 1.0, 33),
    (2, 128256, 0, 0, 1.0, 20), (130, 5003, 1, 2, 3.0, 5), (700, 300, 0, 0, 1.0, 0), (1, 300001, 0, 0, 1.0, 64),
])
def test_parity(dtype, N, V, pad, shift, tau, k):
    z, tok = logits(N, V, dtype, seed=N + V, pad=pad, shift=shift)
    if N > 2:
        tok[1] = -100
    check(z, tok, tau, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("V,k", [(300, 20), (5000, 64), (128256, 20)])
def test_masks(dtype, V, k):
    """-inf words: none left, one left, fewer than k left, the first or last half, every other word; and masks of
    the type's lowest value, which leave a uniform row when they cover it."""
    z, tok = logits(10, V, dtype, seed=V)
    low = torch.finfo(dtype).min
    z[0] = -float("inf")
    for r, few in ((1, 1), (2, 5), (3, k)):
        keep = torch.randperm(V, device="cuda")[:few]
        row = torch.full_like(z[r], -float("inf"))
        row[keep] = z[r, keep]
        z[r] = row
        tok[r] = keep[0]
    z[4, : V // 2] = -float("inf")
    z[5, V // 2:] = -float("inf")
    z[6, ::2] = -float("inf")
    z[7] = low
    z[8, 7:] = low
    z[9, : V - 3] = low
    tok[4] = 0  # a masked token
    tok[8] = 3
    check(z, tok, 1.0, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,k", [(3, 5000, 64), (2, 128256, 20), (3, 65, 64)])
def test_ties_and_orders(dtype, N, V, k):
    """All words equal; two values; rising and falling rows (every word a new maximum); -0 beside +0."""
    z = torch.zeros(6, V, dtype=dtype, device="cuda")
    z[0] = 1.5
    z[1, ::3] = 0.25
    z[2] = torch.linspace(-4, 4, V, device="cuda").to(dtype)
    z[3] = torch.linspace(4, -4, V, device="cuda").to(dtype)
    z[4, 1::2] = -0.0
    z[4] *= 1.0
    z[4, V // 2] = 0.0
    z[5] = -torch.arange(V, device="cuda").remainder(7).to(dtype)
    check(z, torch.arange(6, device="cuda") * 7 % V, 1.0, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,k", [(11, 128256, 20), (700, 20001, 8), (700, 9001, 64), (660, 300, 64)])
@pytest.mark.parametrize("mask", [-float("inf"), -1e4, 0.25])
def test_very_many_equal_words(dtype, N, V, k, mask):
    """One value in almost all words, for a few rows and for more than are at work at once; the others lie above and
    below it, at the start, at the end, next to each other, and fewer or more of them than alternatives."""
    z, tok = logits(N, V, dtype, seed=N + V + k)
    n = torch.arange(N, device="cuda")
    v = torch.arange(V, device="cuda")
    keep = torch.zeros(N, V, dtype=torch.bool, device="cuda")
    for kind, words in ((0, v < 0), (1, v < k - 1), (2, v >= V - k + 1), (3, v % 97 == 5), (4, v < 3 * k), (5, v < 4 * k),
                        (6, (v >= V // 3) & (v < V // 3 + 2 * k)), (7, v == V - 1), (8, v >= V - 100), (9, v < V // 2),
                        (10, v == 0)):
        keep[n % 11 == kind] = words
    z = torch.where(keep, z, torch.full_like(z, mask))
    tok[n % 11 == 8] = V - 1
    check(z, tok, 1.0, k)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,V,k,shift", [(1300, 9001, 20, 1), (1300, 9001, 64, 0), (700, 600, 20, 3), (700, 2000, 64, 0),
                                         (640, 130, 64, 0), (650, 5, 5, 2)])
def test_many_rows_of_every_kind(dtype, N, V, k, shift):
    """More rows than the GPU holds at once, so that rows follow one another in the same blocks: ordinary rows beside
    masked, tied, sorted and constant ones."""
    z, tok = logits(N, V, dtype, seed=N + V, shift=shift)
    z[1::11] = -float("inf")
    z[2::11, : V // 2] = -float("inf")
    z[3::11] = 0.5
    z[4::11] = torch.linspace(-4, 4, V, device="cuda").to(dtype)
    z[5::11] = torch.linspace(4, -4, V, device="cuda").to(dtype)
    z[6::11] = torch.arange(V, device="cuda").remainder(3).to(dtype)
    z[7::11, 3:] = -float("inf")
    tok[8::11] = -100
    check(z, tok, 1.0, k)


def test_rows_of_nan():
    """NaN counts as larger than any number, the lowest index first; every result but the order is NaN."""
    z = torch.randn(700, 3000, device="cuda")
    z[::2, 5:2000] = float("nan")
    z[1::4] = float("nan")
    for N in (3, 700):
        r = token_logprobs(z[:N], torch.zeros(N, dtype=torch.int64, device="cuda"), top_k=30)
        ids = r.top_tokens
        assert torch.equal(ids[0], torch.arange(5, 35, device="cuda")) and torch.equal(ids[1], torch.arange(30, device="cuda"))
        assert torch.equal(ids[2], ids[0]) and torch.isnan(r.top_logprobs[:3]).all() and torch.isnan(r.entropy[:3]).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_very_long_row(dtype):
    """20 million words: groups of many warp loads, and the gradient of the same row."""
    z, tok = logits(2, 20_000_003, dtype, seed=13)
    z[1, :-4] = -float("inf")
    tok[1] = 20_000_001
    check(z, tok, 1.0, 5)


def test_nan_inf_and_tokens_out_of_range():
    z, tok = logits(6, 3000, torch.float32, seed=4)
    z[1, 2500] = float("nan")
    z[2, 10] = float("inf")
    z[3, 20] = -float("nan")
    tok[4] = 3000
    tok[5] = 1 << 40
    r = token_logprobs(z, tok, top_k=3)
    lp = f64(r.logprobs)
    assert np.isnan(lp[[1, 2, 3, 4, 5]]).all() and np.isfinite(lp[0])
    assert np.isnan(f64(r.entropy)[[1, 2, 3]]).all() and np.isfinite(f64(r.entropy)[[0, 4, 5]]).all()
    ids = r.top_tokens.cpu().numpy()
    assert ids[1, 0] == 2500 and ids[2, 0] == 10 and ids[3, 0] == 20
    ref = oo.token_logprobs(f64(z)[[0, 4, 5]], [0, 0, 0], 1.0, 3)
    assert np.array_equal(ids[[0, 4, 5]], ref[3])


def test_large_logits_and_small_temperature():
    z, tok = logits(8, 2000, torch.float32, seed=9, std=200.0)
    check(z, tok, 0.05, 10, grad=False)
    z, tok = logits(8, 2000, torch.float32, seed=10, std=1e4)
    check(z, tok, 1.0, 10, grad=False)


def test_other_layouts():
    """Three dimensions, a transposed view, a broadcast row, a slice of the vocabulary: same results as the copy."""
    z, tok = logits(12, 640, torch.bfloat16, seed=11)
    a = token_logprobs(z.view(3, 4, 640), tok.view(3, 4), top_k=4)
    b = check(z, tok, 1.0, 4)
    assert a.logprobs.shape == (3, 4) and a.top_tokens.shape == (3, 4, 4)
    assert torch.equal(a.logprobs.view(-1), b.logprobs) and torch.equal(a.top_tokens.view(-1, 4), b.top_tokens)
    check(z.t().contiguous().t(), tok, 1.0, 4)
    check(z[3:4].expand(5, 640), tok[:5], 1.0, 4)
    check(z[:, 13:600], tok % 500, 1.0, 4)
    one = token_logprobs(z[0], tok[0], top_k=2)
    assert one.logprobs.shape == () and torch.equal(one.logprobs, b.logprobs[0])
    none = token_logprobs(z[:0], tok[:0], top_k=2)
    assert none.logprobs.shape == (0,) and none.top_tokens.shape == (0, 2)


def test_gradient_of_no_rows_and_of_unused_outputs():
    z, tok = logits(4, 100, torch.float32, seed=2)
    z = z.clone().requires_grad_()
    token_logprobs(z, tok).logprobs.sum().backward()  # an expanded upstream gradient
    assert np.allclose(f64(z.grad), oo.token_logprobs_grad(f64(z), tok.cpu().numpy(), 1.0, np.ones(4), np.zeros(4)),
                       atol=1e-6)
    e = z[:0].detach().requires_grad_()
    token_logprobs(e, tok[:0]).entropy.sum().backward()
    assert e.grad.shape == (0, 100)


def test_second_derivatives_are_refused():
    z = torch.randn(4, 50, device="cuda", requires_grad=True)
    w = torch.randn(4, 50, device="cuda", requires_grad=True)
    tok = torch.zeros(4, dtype=torch.int64, device="cuda")
    dz, = torch.autograd.grad(token_logprobs(z, tok).logprobs.sum(), z, create_graph=True)
    plain, = torch.autograd.grad(token_logprobs(z, tok).logprobs.sum(), z)
    assert torch.equal(dz, plain)
    with pytest.raises(RuntimeError, match="differentiable once"):
        (dz * w).sum().backward()
    h, W = (torch.randn(n, 16, device="cuda").bfloat16().requires_grad_() for n in (4, 50))
    grads = torch.autograd.grad(head_logprobs(h, W, tok)[0].sum(), (h, W), create_graph=True)
    for g in grads:
        with pytest.raises(RuntimeError, match="differentiable once"):
            g.float().sum().backward(retain_graph=True)


def test_gradient_against_differences():
    """d/dz from the kernel against central differences of the fp64 forward: error of the differences 1e-9,
    of the fp32 gradient 1e-6 of its size (at most 4)."""
    z, tok = logits(3, 11, torch.float32, seed=5)
    tau, gl, ge = 0.8, np.array([1.0, -0.5, 2.0]), np.array([0.3, 1.0, -1.0])
    z = z.requires_grad_()
    r = token_logprobs(z, tok, tau=tau)
    g = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    dz, = torch.autograd.grad((r.logprobs, r.entropy), (z,), (g(gl), g(ge)))
    x = f64(z)

    def f(y):
        lp, H, _, _ = oo.token_logprobs(y, tok.cpu().numpy(), tau)
        return (gl * lp + ge * H).sum()

    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1e-5
        assert abs((f(x + e) - f(x - e)) / 2e-5 - f64(dz)[i]) < 4e-6


def test_repeatable_in_place_and_on_another_stream():
    z, tok = logits(40, 9001, torch.bfloat16, seed=6)
    a = token_logprobs(z, tok, top_k=9)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        z2 = z * 1.0
        b = token_logprobs(z2, tok, top_k=9)
    s.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    f = dict(dtype=torch.float32, device="cuda")
    lp, H, st = torch.empty(40, **f), torch.empty(40, **f), torch.empty(40, 2, **f)
    g = torch.randn(40, **f)
    zc = z.clone()  # contiguous rows of 9001 elements
    _lib.hylo_token_logprobs(zc, tok, 1.0, 0, lp, H, None, st)
    out = torch.empty_like(zc)
    _lib.hylo_token_logprobs_backward(zc, tok, 1.0, st, H, g, g, out)
    _lib.hylo_token_logprobs_backward(zc, tok, 1.0, st, H, g, g, zc)  # over the logits themselves
    assert torch.equal(out, zc)
    odd = torch.empty(40, 9004, dtype=z.dtype, device="cuda")[:, 3:]  # rows at other offsets than the logits'
    _lib.hylo_token_logprobs_backward(z, tok, 1.0, st, H, g, g, odd)
    assert torch.equal(out, odd)
    zero = torch.full_like(out, 1.0)
    _lib.hylo_token_logprobs_backward(z, tok, 1.0, st, None, None, None, zero)
    assert torch.all(zero == 0)


def test_graph_capture():
    z, tok = logits(9, 4000, torch.bfloat16, seed=8)
    z = z.clone()
    token_logprobs(z, tok, top_k=5)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r = token_logprobs(z, tok, top_k=5)
    z.copy_(logits(9, 4000, torch.bfloat16, seed=88)[0])
    g.replay()
    e = token_logprobs(z, tok, top_k=5)
    for x, y in zip(r, e):
        assert torch.equal(x, y)


def test_rows_behind_2_to_31_elements():
    """Row offsets that pass 32 bits: 20000 rows of 128256 words (5.1 GB), the last ones checked."""
    N, V = 20000, 128256
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    part, _ = logits(4, V, torch.bfloat16, seed=12)
    z[-4:] = part
    tok = torch.full((N,), V - 1, dtype=torch.int64, device="cuda")
    r = token_logprobs(z, tok, top_k=4)
    lp, H, top, ids = oo.token_logprobs(f64(part), tok[-4:].cpu().numpy(), 1.0, 4)
    near(r.logprobs[-4:], lp, (V / 256 + 96) * U)
    assert np.array_equal(r.top_tokens[-4:].cpu().numpy(), ids)
    assert np.array_equal(r.top_tokens[N // 2].cpu().numpy(), np.arange(4))
