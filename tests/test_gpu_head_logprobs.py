"""GPU parity of head_logprobs (forward and gradients) against the fp64 oracle.

Tolerances: a logit is an fp32 sum of d products accumulated 16 at a time, off by at most (d/16) 2^-23 of
sum |h W|, taken here as the logits' scale times sqrt(d) (inputs are of random signs): dz = 2^-23 (d/16 + 8)
max|z|. logp and entropy take that, the softmax sums' (V/256 + 64) 2^-24 (1 + |x|) and nothing else. Gradients:
G rounded to bf16 once is within 2^-8 of each element, at random, so 4e-3 of the norm bounds dh and dW
also where few elements dominate; with split_g 2^-16 and the fp32 sums remain: 1e-4. Autograd
results are rounded to bf16 once more: another 2^-8.
"""
import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, head_logprobs, token_logprobs
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def f64(t):
    return t.detach().double().cpu().numpy()


def inputs(N, d, V, seed=0, std=1.3):
    gen = torch.Generator("cuda").manual_seed(seed)
    h = torch.randn(N, d, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, d, generator=gen, device="cuda") * (std / d ** 0.5)).bfloat16()
    tok = torch.randint(0, V, (N,), generator=gen, device="cuda")
    if N > 4:
        tok[2], tok[4] = -100, V - 1
    return h, W, tok


def near(x, ref, tol):
    err = np.abs(f64(x) - ref) / (1 + np.abs(ref))
    assert err.max() <= tol, (err.max(), tol)


def tol_of(z, d, V, tau):
    return (V / 256 + 64) * 2.0 ** -24 + 2.0 ** -22 * (d / 16 + 8) * np.abs(z).max() / tau


@pytest.mark.parametrize("N,d,V,tau", [
    (1, 8, 1, 1.0), (1, 64, 300, 0.5), (3, 72, 257, 1.0), (130, 520, 1000, 2.0), (257, 128, 255, 1.0), (300, 256, 5003, 1.0),
    (1, 2048, 128256, 1.0), (5, 4096, 33001, 0.7), (600, 2048, 2050, 1.0), (1025, 64, 40000, 1.0),
])
def test_forward(N, d, V, tau):
    h, W, tok = inputs(N, d, V, seed=N + d)
    logp, ent = head_logprobs(h, W, tok, tau=tau)
    z = f64(h) @ f64(W).T
    lp, H, _, _ = oo.token_logprobs(z, tok.cpu().numpy(), tau)
    near(logp, lp, tol_of(z, d, V, tau))
    near(ent, H, 2 * tol_of(z, d, V, tau))


@pytest.mark.parametrize("N,d,V", [(3, 2048, 20_001), (8, 4096, 9000), (15, 4096, 8193), (31, 2048, 16_400), (32, 2048, 16_400),
                                   (5, 65536, 600), (3, 16, 2_100_003)])
def test_few_tokens_of_a_large_head(N, d, V):
    """A head of 64 MiB and more with hidden states of less than 128 KiB, or just that; also in a larger batch."""
    h, W, tok = inputs(N, d, V, seed=N)
    logp, ent = head_logprobs(h, W, tok)
    z = f64(h) @ f64(W).T
    lp, H, _, _ = oo.token_logprobs(z, tok.cpu().numpy(), 1.0)
    near(logp, lp, tol_of(z, d, V, 1.0))
    near(ent, H, 2 * tol_of(z, d, V, 1.0))
    many, _ = head_logprobs(h.repeat(40, 1), W, tok.repeat(40))
    near(many.view(40, N)[7], lp, tol_of(z, d, V, 1.0))


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("N,d,V,tau,chunk", [
    (1, 8, 3, 1.0, 0), (5, 72, 300, 0.5, 4096), (130, 520, 1000, 2.0, 4096), (700, 256, 5003, 1.0, 256),
    (300, 2048, 20000, 1.0, 4096), (1500, 64, 9001, 0.8, 512),
])
def test_gradients(N, d, V, tau, chunk, split):
    h, W, tok = inputs(N, d, V, seed=N)
    rng = np.random.default_rng(N)
    gl, ge = rng.normal(size=N), 0.3 * rng.normal(size=N)
    t = lambda x: torch.tensor(x, dtype=torch.float32, device="cuda")  # noqa: E731
    h.requires_grad_(), W.requires_grad_()
    logp, ent = head_logprobs(h, W, tok, tau=tau, token_chunk=chunk, split_g=split)
    z = f64(h) @ f64(W).T
    for a, b in ((gl, ge), (gl, None), (None, ge)):
        pairs = [(o, t(g)) for o, g in ((logp, a), (ent, b)) if g is not None]
        dh, dW = torch.autograd.grad([o for o, _ in pairs], (h, W), [g for _, g in pairs], retain_graph=True)
        G = oo.token_logprobs_grad(z, tok.cpu().numpy(), tau, np.zeros(N) if a is None else a, np.zeros(N) if b is None else b)
        for got, ref in ((dh, G @ f64(W)), (dW, G.T @ f64(h))):
            bound = ((1e-4 if split else 4e-3) + 2.0 ** -8) * np.linalg.norm(ref) + 1e-5 * np.abs(gl).max()
            assert got.dtype == torch.bfloat16 and np.linalg.norm(f64(got) - ref) <= bound


@pytest.mark.parametrize("split,tol", [(False, 4e-3), (True, 1e-4)])
def test_fp32_gradients_of_the_c_abi(split, tol):
    N, d, V, tau = 400, 512, 3000, 1.0
    h, W, tok = inputs(N, d, V, seed=4)
    f = dict(dtype=torch.float32, device="cuda")
    lp, H, lse = (torch.empty(N, **f) for _ in range(3))
    ws = torch.empty(_lib.hylo_head_logprobs_workspace_bytes(N, d, V, 256, split), dtype=torch.uint8, device="cuda")
    _lib.hylo_head_logprobs(h, W, tok, tau, lp, H, lse, ws)
    g = torch.randn(N, **f)
    dh, dW = torch.full((N, d), float("nan"), **f), torch.full((V, d), float("nan"), **f)
    _lib.hylo_head_logprobs_backward(h, W, tok, tau, 256, lse, H, g, g, dh, dW, ws, split)
    _lib.hylo_kl_sync_status()
    G = oo.token_logprobs_grad(f64(h) @ f64(W).T, tok.cpu().numpy(), tau, f64(g), f64(g))
    for got, ref in ((dh, G @ f64(W)), (dW, G.T @ f64(h))):
        assert np.linalg.norm(f64(got) - ref) <= tol * np.linalg.norm(ref)
    b = dict(dtype=torch.bfloat16, device="cuda")
    for chunk in (256, 4096):  # bf16 gradients are the fp32 ones rounded: by a pass of their own, or at once (one token block)
        wb = torch.empty(_lib.hylo_head_logprobs_workspace_bytes(N, d, V, chunk, split, torch.bfloat16), dtype=torch.uint8,
                         device="cuda")
        f_h, f_W, b_h, b_W = torch.empty(N, d, **f), torch.empty(V, d, **f), torch.empty(N, d, **b), torch.empty(V, d, **b)
        _lib.hylo_head_logprobs_backward(h, W, tok, tau, chunk, lse, H, g, g, f_h, f_W, wb, split)
        _lib.hylo_head_logprobs_backward(h, W, tok, tau, chunk, lse, H, g, g, b_h, b_W, wb, split)
        assert torch.equal(b_h, f_h.bfloat16()) and torch.equal(b_W, f_W.bfloat16())
    again_h, again_W = torch.empty_like(dh), torch.empty_like(dW)
    _lib.hylo_head_logprobs_backward(h, W, tok, tau, 256, lse, H, g, g, again_h, again_W, ws, split)
    assert torch.equal(dh, again_h) and torch.equal(dW, again_W)


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("N,d,V", [(300, 64, 100_000), (700, 64, 60_001), (1, 128, 200_001), (1000, 72, 150_007)])
def test_gradients_over_many_vocabulary_blocks(N, d, V, split):
    """Few tokens and many vocabulary blocks, so that G's buffers are used again: the bound of test_gradients, taken
    also over each stretch of 8192 words and each token alone (1.5 times: fewer elements to average over for a token)."""
    h, W, tok = inputs(N, d, V, seed=V)
    tok[0] = V - 1
    gl, ge = torch.randn(N, device="cuda"), 0.3 * torch.randn(N, device="cuda")
    h.requires_grad_(), W.requires_grad_()
    logp, ent = head_logprobs(h, W, tok, split_g=split)
    dh, dW = torch.autograd.grad([logp, ent], (h, W), [gl, ge])
    G = oo.token_logprobs_grad(f64(h) @ f64(W).T, tok.cpu().numpy(), 1.0, f64(gl), f64(ge))
    rel = (1e-4 if split else 4e-3) + 2.0 ** -8
    ref_h, ref_W = G @ f64(W), G.T @ f64(h)
    for n in range(N):
        assert np.linalg.norm(f64(dh[n]) - ref_h[n]) <= 1.5 * rel * np.linalg.norm(ref_h[n]) + 1e-5 * gl.abs().max().item()
    for v in range(0, V, 8192):
        ref = ref_W[v:v + 8192]
        assert np.linalg.norm(f64(dW[v:v + 8192]) - ref) <= rel * np.linalg.norm(ref) + 1e-5 * gl.abs().max().item()


@pytest.mark.parametrize("N,d,V,chunk", [(1500, 64, 60_001, 4096), (1100, 72, 200_001, 256), (600, 64, 100_001, 256)])
def test_gradients_over_blocks_of_tokens_and_words(N, d, V, chunk):
    """Sums over vocabulary blocks (dh) and over token blocks (dW) one after another: five vocabulary blocks of all
    tokens; five token blocks by three vocabulary blocks; three by two. Bounds as above; and bitwise the same again."""
    h, W, tok = inputs(N, d, V, seed=V)
    gl, ge = torch.randn(N, device="cuda"), 0.3 * torch.randn(N, device="cuda")
    h.requires_grad_(), W.requires_grad_()
    logp, ent = head_logprobs(h, W, tok, token_chunk=chunk)
    dh, dW = torch.autograd.grad([logp, ent], (h, W), [gl, ge], retain_graph=True)
    for _ in range(3):
        again = torch.autograd.grad([logp, ent], (h, W), [gl, ge], retain_graph=True)
        assert torch.equal(dh, again[0]) and torch.equal(dW, again[1])
    G = oo.token_logprobs_grad(f64(h) @ f64(W).T, tok.cpu().numpy(), 1.0, f64(gl), f64(ge))
    rel = 4e-3 + 2.0 ** -8
    ref_h, ref_W = G @ f64(W), G.T @ f64(h)
    for n in range(N):
        assert np.linalg.norm(f64(dh[n]) - ref_h[n]) <= 1.5 * rel * np.linalg.norm(ref_h[n]) + 1e-5 * gl.abs().max().item()
    for v in range(0, V, 8192):
        ref = ref_W[v:v + 8192]
        assert np.linalg.norm(f64(dW[v:v + 8192]) - ref) <= rel * np.linalg.norm(ref) + 1e-5 * gl.abs().max().item()


@pytest.mark.parametrize("N,d,V,chunk,split", [(300, 64, 100_000, 4096, False), (1500, 64, 60_001, 4096, False),
                                               (1100, 72, 200_001, 256, False), (600, 64, 5000, 256, True), (40, 512, 3000, 4096, None)])
def test_one_gradient_alone_is_that_of_both(N, d, V, chunk, split):
    """Frozen hidden states or a frozen LM head: the other gradient, bit for bit; fp32 through the C ABI too."""
    h, W, tok = inputs(N, d, V, seed=N)
    gl, ge = torch.randn(N, device="cuda"), torch.randn(N, device="cuda")

    def grads(*need):
        hh, WW = h.detach().clone(), W.detach().clone()
        for t, n in zip((hh, WW), need):
            t.requires_grad_(n)
        out = head_logprobs(hh, WW, tok, token_chunk=chunk, split_g=split)
        (out[0] @ gl + out[1] @ ge).backward()
        return hh.grad, WW.grad

    dh, dW = grads(True, True)
    only_h, only_W = grads(True, False), grads(False, True)
    assert torch.equal(dh, only_h[0]) and only_h[1] is None and torch.equal(dW, only_W[1]) and only_W[0] is None
    f = dict(dtype=torch.float32, device="cuda")
    lp, H, lse = (torch.empty(N, **f) for _ in range(3))
    ws = torch.empty(_lib.hylo_head_logprobs_workspace_bytes(N, d, V, chunk, bool(split)), dtype=torch.uint8, device="cuda")
    _lib.hylo_head_logprobs(h, W, tok, 1.0, lp, H, lse, ws)
    both = torch.empty(N, d, **f), torch.empty(V, d, **f)
    _lib.hylo_head_logprobs_backward(h, W, tok, 1.0, chunk, lse, H, gl, ge, *both, ws, bool(split))
    for k in range(2):
        one = torch.full_like(both[k], float("nan"))
        _lib.hylo_head_logprobs_backward(h, W, tok, 1.0, chunk, lse, H, gl, ge, *((one, None) if k == 0 else (None, one)), ws,
                                         bool(split))
        _lib.hylo_kl_sync_status()
        assert torch.equal(one, both[k])


def test_gradient_against_differences():
    """Directional differences of the fp64 forward along random directions; bound: G's one rounding to bf16."""
    N, d, V = 6, 16, 40
    h, W, tok = inputs(N, d, V, seed=3)
    h.requires_grad_(), W.requires_grad_()
    gl = np.linspace(-1, 1, N)
    logp, ent = head_logprobs(h, W, tok, split_g=True)
    (logp * torch.tensor(gl, dtype=torch.float32, device="cuda")).sum().add(ent.sum()).backward()
    hn, Wn, tn = f64(h), f64(W), tok.cpu().numpy()

    def f(a, b):
        lp, H, _, _ = oo.token_logprobs(a @ b.T, tn)
        return (gl * lp + H).sum()

    rng = np.random.default_rng(0)
    for _ in range(5):
        u, v = rng.normal(size=hn.shape), rng.normal(size=Wn.shape)
        e = 1e-5
        diff = (f(hn + e * u, Wn + e * v) - f(hn - e * u, Wn - e * v)) / (2 * e)
        mine = (f64(h.grad) * u).sum() + (f64(W.grad) * v).sum()
        size = np.linalg.norm(f64(h.grad)) * np.linalg.norm(u) + np.linalg.norm(f64(W.grad)) * np.linalg.norm(v)
        assert abs(diff - mine) <= (2.0 ** -8 + 1e-4) * size


def test_layouts_streams_and_the_logits_operator():
    h, W, tok = inputs(24, 128, 700, seed=7)
    a = head_logprobs(h, W, tok)
    b = head_logprobs(h.view(4, 6, 128), W, tok.view(4, 6))
    assert b[0].shape == (4, 6) and torch.equal(a[0], b[0].view(-1)) and torch.equal(a[1], b[1].view(-1))
    wide = torch.randn(24, 200, device="cuda").bfloat16()
    wide[:, :128] = h
    c = head_logprobs(wide[:, :128], W.t().contiguous().t(), tok)
    assert torch.equal(a[0], c[0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        e = head_logprobs(h, W, tok)
    s.synchronize()
    assert torch.equal(a[0], e[0]) and torch.equal(a[1], e[1])
    r = token_logprobs(h.float() @ W.float().T, tok)
    assert torch.allclose(r.logprobs, a[0], atol=1e-4) and torch.allclose(r.entropy, a[1], atol=1e-4)
    one = head_logprobs(h[0], W, tok[0])
    assert one[0].shape == () and torch.allclose(one[0], a[0][0], atol=1e-5)  # another split of the vocabulary
    empty = head_logprobs(h[:0], W, tok[:0])
    assert empty[0].shape == (0,)
    bad = tok.clone()
    bad[3], bad[5] = 700, 1 << 40
    x = head_logprobs(h, W, bad)[0]
    assert torch.isnan(x[[3, 5]]).all() and torch.isfinite(x).sum() == 22


def test_graph_capture():
    h, W, tok = inputs(50, 256, 3000, seed=9)
    f = dict(dtype=torch.float32, device="cuda")
    lp, H, lse = (torch.empty(50, **f) for _ in range(3))
    dh, dW, g = torch.empty(50, 256, **f), torch.empty(3000, 256, **f), torch.randn(50, **f)
    ws = torch.empty(_lib.hylo_head_logprobs_workspace_bytes(50, 256, 3000), dtype=torch.uint8, device="cuda")

    def step():
        _lib.hylo_head_logprobs(h, W, tok, 1.0, lp, H, lse, ws)
        _lib.hylo_head_logprobs_backward(h, W, tok, 1.0, 4096, lse, H, g, None, dh, dW, ws)

    step()
    want = [x.clone() for x in (lp, H, lse, dh, dW)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x in (lp, H, lse, dh, dW):
        x.zero_()
    graph.replay()
    graph.replay()
    for x, y in zip((lp, H, lse, dh, dW), want):
        assert torch.equal(x, y)


def test_first_cuda_call_of_a_thread():
    """A call from a thread that has made no CUDA call before (as autograd's workers do)."""
    import threading
    h, W, tok = inputs(20, 64, 500, seed=2)
    f = dict(dtype=torch.float32, device="cuda")
    lp, H, lse = (torch.empty(20, **f) for _ in range(3))
    dh, dW, g = torch.empty(20, 64, **f), torch.empty(500, 64, **f), torch.ones(20, **f)
    ws = torch.empty(_lib.hylo_head_logprobs_workspace_bytes(20, 64, 500), dtype=torch.uint8, device="cuda")
    _lib.hylo_head_logprobs(h, W, tok, 1.0, lp, H, lse, ws)
    stream, errors = torch.cuda.current_stream().cuda_stream, []

    def work():
        st = _lib.load().hylo_head_logprobs_backward(
            h.data_ptr(), W.data_ptr(), 20, 64, 500, 1.0, 0, tok.data_ptr(), lse.data_ptr(), None, g.data_ptr(), None, 0, 0,
            dh.data_ptr(), dW.data_ptr(), ws.data_ptr(), ws.numel(), stream)
        errors.append(st)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert errors == [0]
    G = oo.token_logprobs_grad(f64(h) @ f64(W).T, tok.cpu().numpy(), 1.0, np.ones(20), np.zeros(20))
    assert np.linalg.norm(f64(dh) - G @ f64(W)) <= 4e-3 * np.linalg.norm(G @ f64(W))


def test_large_shape_rows_against_float64():
    """The 1B student's head over 4096 tokens, 64 rows of each result against float64 on the device."""
    N, d, V = 4096, 2048, 128256
    h, W, tok = inputs(N, d, V, seed=1)
    h.requires_grad_(), W.requires_grad_()
    logp, ent = head_logprobs(h, W, tok)
    g = torch.randn(N, device="cuda")
    dh, dW = torch.autograd.grad((logp, ent), (h, W), (g, 0.1 * g))
    with torch.no_grad():
        pick = torch.arange(0, N, 64, device="cuda")
        Wd = W.double()
        z = h[pick].double() @ Wd.T
        lp, H, _, _ = oo.token_logprobs(f64(z), tok[pick].cpu().numpy())
        near(logp[pick], lp, tol_of(f64(z), d, V, 1.0))
        near(ent[pick], H, 2 * tol_of(f64(z), d, V, 1.0))
        G = torch.tensor(oo.token_logprobs_grad(f64(z), tok[pick].cpu().numpy(), 1.0, f64(g[pick]), f64(0.1 * g[pick])), device="cuda")
        ref = G @ Wd
        assert (dh[pick].double() - ref).norm() <= (4e-3 + 2.0 ** -8) * ref.norm()
        words = torch.arange(5, V, 2004, device="cuda")  # all tokens' part of these words' gradient
        z = h.double() @ Wd.T
        llp = torch.log_softmax(z, 1)
        Hall = -(llp.exp() * llp).sum(1, keepdim=True)
        part = llp[:, words]
        a, b = (g * (tok >= 0)).double()[:, None], (0.1 * g).double()[:, None]
        Gw = a * ((tok[:, None] == words) * 1.0 - part.exp()) - b * part.exp() * (part + Hall)
        ref = Gw.T @ h.double()
        assert (dW[words].double() - ref).norm() <= (4e-3 + 2.0 ** -8) * ref.norm()
