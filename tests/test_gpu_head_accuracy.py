"""Log-probabilities from deep hidden states: the drift of the tensor cores' accumulation does not grow with d.

Tolerance: a logit is accumulated over at most 64 steps of 16 products before its parts are added up, each step off by at most
2^-23 of the partial sum, so 2^-22 (64 + 8) max|z| for logp and its normaliser together, as in the other tests of the operator
with d / 16 = 64, and the softmax sums' (V / 256 + 64) 2^-24 (1 + |x|).
"""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, head_logprobs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


@pytest.mark.parametrize("d", [1024, 1032, 2048, 16384, 65536])
@pytest.mark.parametrize("N,V", [(1, 600), (3, 600), (300, 257), (3, 5003)])
@pytest.mark.parametrize("train", [False, True])
def test_logits_that_grow_all_along_d(N, V, d, train):
    """Every product of the token's logit has the same sign, the sum that drifts most, and its probability is small, so that the
    normaliser does not drift with it."""
    gen = torch.Generator("cuda").manual_seed(N + d)
    W = (torch.randn(V, d, generator=gen, device="cuda") / d ** 0.5).bfloat16()
    t = torch.randint(0, V, (N,), generator=gen, device="cuda")
    h = (torch.randn(N, d, generator=gen, device="cuda") * 0.3 + 5.0 * W[t].float()).bfloat16()
    h.requires_grad_(train)
    logp, ent = head_logprobs(h, W, t)
    z = h.detach().double() @ W.double().T
    lp = torch.log_softmax(z, 1)
    top = z.abs().max().item()
    for got, ref, k in ((logp, lp.gather(1, t[:, None])[:, 0], 1), (ent, torch.special.entr(lp.exp()).sum(1), 2)):
        tol = k * ((V / 256 + 64) * 2.0 ** -24 * (1 + ref.abs()) + 2.0 ** -22 * 72 * top)
        assert torch.all((got.double() - ref).abs() <= tol)
    if train:
        dh, = torch.autograd.grad(logp.sum(), h)
        G = -lp.exp()
        G.scatter_add_(1, t[:, None], torch.ones_like(logp, dtype=torch.float64)[:, None])
        ref = G @ W.double()
        assert ((dh.double() - ref).norm() / ref.norm()).item() <= 4e-3 + 2.0 ** -8
    _lib.hylo_kl_sync_status()
