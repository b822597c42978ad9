"""orthogonalize has no derivatives: they are refused where they are asked for, not dropped."""
import pytest
import torch
from torch.autograd import forward_ad

from hybrid_upcycling_gb300 import build, orthogonalize


def test_tangents_are_refused():
    x = torch.randn(4, 6)
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for mats in (dual, [x, dual]):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                orthogonalize(mats)


@pytest.mark.gpu
def test_a_backward_through_a_result_is_refused():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    x, w = torch.randn(40, 60, device="cuda"), torch.randn(60, 40, device="cuda", requires_grad=True)
    plain = orthogonalize([x, w.detach(), w.detach().mT])
    for y in (orthogonalize(w), orthogonalize([x, w])[1], orthogonalize([w.mT])[0].mT, orthogonalize((2 * w).view(1, 60, 40))[0]):
        with pytest.raises(RuntimeError, match="orthogonalize is not differentiable"):
            (y.float() * w).sum().backward()
    assert w.grad is None
    got = orthogonalize([x, w, w.mT])
    assert all(torch.equal(a, b) for a, b in zip(got, plain))       # the same results
    assert not got[0].requires_grad and all(t.requires_grad and t.is_contiguous() for t in got[1:])
    got[1].mul_(2)                                                  # which may be written in place
    assert torch.equal(got[1], 2 * plain[1])
    with torch.no_grad():
        assert not orthogonalize(w).requires_grad
    (w * orthogonalize(w).detach()).sum().backward()                # as a constant
    assert torch.equal(w.grad, plain[1].float())
