"""Gradients of tokens that the model is nearly sure of: G = g (1 - p) of the token is a difference, so the probabilities that the
backward computes again have to be those of the forward's lse.

Tolerance, u = 2^-24: with |lse| <= L the backward's log2(e) (z - lse) takes lse rounded (L u), its product with log2(e) rounded
(2 L u), the multiply-add's rounding and ex2.approx (4 u), and lse the error of log s, (V / 256 + 64) u / 8 at most for sums of
random rounding errors: an absolute error of p of at most D = (3 L + 4 + (V / 256 + 64) / 8) u, relative to 1 - p. With
the split G and fp32 gradients 1e-4 of the norm besides, as in the other tests; G in bf16 4e-3.
"""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def confident(N, d, V, gap, gen):
    """h, W, tokens with z_token = log(sum of the others' e^z) + gap."""
    W = (torch.randn(V, d, generator=gen, device="cuda") * 0.02).bfloat16()
    t = torch.randint(0, V, (N,), generator=gen, device="cuda")
    h, w = torch.randn(N, d, generator=gen, device="cuda").double(), W[t].double()
    z = h @ W.double().T
    others = torch.logsumexp(z.scatter(1, t[:, None], -float("inf")), 1, keepdim=True)
    h = h + (others + gap - z.gather(1, t[:, None])) * w / (w * w).sum(1, keepdim=True)
    return h.bfloat16(), W, t


@pytest.mark.parametrize("N", [1, 2, 3, 64, 256, 300])
@pytest.mark.parametrize("d,V", [(512, 5003), (2048, 20000), (4096, 9000)])
@pytest.mark.parametrize("gap", [2.0, 7.0])
@pytest.mark.parametrize("split", [True, False])
def test_gradient(N, d, V, gap, split):
    gen = torch.Generator("cuda").manual_seed(N + d)
    h, W, t = confident(N, d, V, gap, gen)
    f = dict(dtype=torch.float32, device="cuda")
    logp, ent, lse = (torch.empty(N, **f) for _ in range(3))
    ws = torch.empty(_lib.hylo_head_logprobs_workspace_bytes(N, d, V, 4096, split), dtype=torch.uint8, device="cuda")
    _lib.hylo_head_logprobs(h, W, t, 1.0, logp, ent, lse, ws)
    dh, dW, g = torch.empty(N, d, **f), torch.empty(V, d, **f), torch.ones(N, **f)
    _lib.hylo_head_logprobs_backward(h, W, t, 1.0, 4096, lse, ent, g, None, dh, dW, ws, split)
    _lib.hylo_kl_sync_status()
    hd, Wd = h.double(), W.double()
    p = torch.softmax(hd @ Wd.T, 1)
    rest = p.scatter(1, t[:, None], 0.0).sum(1, keepdim=True)  # 1 - p
    G = -p.scatter(1, t[:, None], -rest)
    D = (3 * lse.abs().max().item() + 4 + (V / 256 + 64) / 8) * 2.0 ** -24
    tol = (1e-4 if split else 4e-3) + D / rest.min().item()
    for got, ref in ((dh, G @ Wd), (dW, G.T @ hd)):
        assert ((got.double() - ref).norm() / ref.norm()).item() <= tol
