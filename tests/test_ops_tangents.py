"""Forward-mode derivatives are refused, not dropped: a dual tensor raises whether or not it also asks for a gradient."""
import pytest
import torch
from torch.autograd import forward_ad

from hybrid_upcycling_gb300 import head_logprobs, token_logprobs


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
@pytest.mark.parametrize("requires_grad", [False, True])
@pytest.mark.parametrize("no_grad", [False, True])
def test_dual_tensors_are_refused(device, requires_grad, no_grad):
    if device == "cuda" and not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    t = torch.zeros(3, dtype=torch.int64, device=device)
    z, h, W = (torch.randn(n, m, device=device) for n, m in ((3, 16), (3, 16), (10, 16)))
    h, W = h.bfloat16(), W.bfloat16()
    for x in (z, h, W):
        x.requires_grad_(requires_grad)
    with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
        dual = [forward_ad.make_dual(x, torch.ones_like(x)) for x in (z, h, W)]
        for call in (lambda: token_logprobs(dual[0], t), lambda: token_logprobs(dual[0][None], t[None], top_k=2),
                     lambda: head_logprobs(dual[1], W, t), lambda: head_logprobs(h, dual[2], t)):
            with pytest.raises(NotImplementedError):
                call()
    if device == "cuda":
        assert torch.isfinite(token_logprobs(z.detach(), t).logprobs).all()
