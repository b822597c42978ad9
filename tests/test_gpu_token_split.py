"""token_logprobs of rows that a cluster shares, where the last CTAs of the cluster have no words and the row ends inside a
group: its best words are put into that last group, for one row and for several rows one after another in a cluster.

Tolerance of the log-probabilities: as in the other tests of the operator, (V / 256 + 96) 2^-24 (1 + |x|).
"""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, token_logprobs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


@pytest.mark.parametrize("dtype,V,rows", [
    (torch.bfloat16, 151936, (1, 2, 7, 32)), (torch.float32, 151936, (1, 3, 32)), (torch.float16, 135300, (1, 5, 30)),
    (torch.bfloat16, 135300, (1, 16)), (torch.float32, 32768, (1, 9)), (torch.float32, 300001, (2,)),
    (torch.float32, 1_000_001, (70, 110, 200)), (torch.bfloat16, 2_000_003, (110,))])
def test_best_words_at_the_end(dtype, V, rows):
    k = 13
    gen = torch.Generator("cuda").manual_seed(V)
    for N in rows:
        z = torch.empty(N, V, dtype=dtype, device="cuda")
        for r in range(N):
            z[r] = torch.randn(V, generator=gen, device="cuda").clamp(-3, 3)
        # distinct values above all others, within the last 40 words, in an order of each row's own
        place = torch.stack([torch.randperm(40, generator=gen, device="cuda")[:k] for _ in range(N)]) + (V - 40)
        best = (12.0 - 0.25 * torch.arange(k, device="cuda")).to(dtype).expand(N, k)
        z.scatter_(1, place, best)
        for _ in range(3):
            r = token_logprobs(z, place[:, 0].contiguous(), top_k=k)
            assert torch.equal(r.top_tokens, place)
        for lo in range(0, N, 16):
            lse = torch.logsumexp(z[lo:lo + 16].double(), 1, keepdim=True)
            ref = best[lo:lo + 16].double() - lse
            err = (r.top_logprobs[lo:lo + 16].double() - ref).abs() / (1 + ref.abs())
            assert err.max() <= (V / 256 + 96) * 2.0 ** -24
            assert torch.equal(r.logprobs[lo:lo + 16], r.top_logprobs[lo:lo + 16, 0])
