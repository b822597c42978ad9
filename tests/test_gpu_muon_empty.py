"""Batches without elements, of any number of dimensions, are results without elements."""
import pytest
import torch

from hybrid_upcycling_gb300 import build, muon_step, orthogonalize

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(2, 3, 0, 5), (2, 3, 5, 0), (0, 3, 5, 4), (2, 0, 5, 4), (2, 3, 0, 0), (1, 2, 3, 0, 7), (3, 0, 5), (0, 5), (5, 0)])
def test_batches_without_elements(shape):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    x = torch.empty(shape, device="cuda")
    full = torch.randn(20, 30, device="cuda")
    y = orthogonalize(x)
    assert y.shape == x.shape and y.dtype == torch.bfloat16 and y.is_contiguous()
    turned = orthogonalize(x.transpose(-1, -2))
    assert turned.shape == x.transpose(-1, -2).shape and turned.is_contiguous()
    alone = orthogonalize(full)
    a, b, c = orthogonalize([full, x, full.mT])  # beside matrices that have some
    assert torch.equal(a, alone) and b.shape == x.shape and torch.equal(c, alone.mT)
    muon_step([x], [x.clone()], [torch.empty(shape, device="cuda")], lr=0.1)
