"""8-bit states need an eps that the kernel's arithmetic does not take for 0 (an element without gradient or moments: 0 / 0)."""
import struct

import pytest
import torch

from hybrid_upcycling_gb300 import State8, _lib, adamw_step, build

FAKE = 0x100000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("eps", [0.0, 1e-300, 1e-45, 1e-39, 1.17e-38])
def test_a_subnormal_eps_is_refused(lib, eps):
    table = struct.pack("=" + _lib.ADAMW_TENSOR, *(FAKE + 0x1000 * i for i in range(2)), 0, *(FAKE + 0x1000 * i for i in range(3, 7)),
                        10, 1e-3, 0.1)
    assert lib.hylo_adamw_step(table, 1, 0, 0, 8, 0.9, 0.999, eps, 1, 1.0, None, 1.0, 0, None) == -2
    assert b"eps" in lib.hylo_kl_last_error()


@pytest.mark.gpu
def test_the_smallest_eps_leaves_elements_without_gradient_alone(lib):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    p, g = torch.ones(3000, device="cuda"), torch.zeros(3000, device="cuda")
    adamw_step([p], [g], [State8.zeros_like(p)], [State8.zeros_like(p)], step=1, lr=0.1, eps=2.0 ** -126, weight_decay=0.5)
    assert torch.all((p - 0.95).abs() < 1e-6)
