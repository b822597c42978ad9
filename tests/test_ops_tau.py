"""A temperature so small that log2(e) / tau is infinite is refused by every entry point: the kernels would work with 0 * inf."""
import pytest

from hybrid_upcycling_gb300 import _lib, build

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


@pytest.mark.parametrize("tau", [3e-39, 3.5e-39, 4.2e-39])  # 1 / tau is finite
def test_tau_below_the_kernels_range(lib, tau):
    n = 1 << 30
    assert lib.hylo_token_logprobs(FAKE, 1, 4, 100, 100, tau, FAKE, 5, FAKE, FAKE, None, FAKE, FAKE, FAKE, None) == -4
    assert lib.hylo_token_logprobs_backward(FAKE, 1, 4, 100, 100, tau, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 100, None) == -4
    assert lib.hylo_head_logprobs(FAKE, FAKE, 16, 64, 100, tau, FAKE, FAKE, None, None, FAKE, n, None) == -4
    assert lib.hylo_head_logprobs_backward(FAKE, FAKE, 16, 64, 100, tau, 0, FAKE, FAKE, FAKE, FAKE, FAKE, 0, 0, FAKE, FAKE, FAKE,
                                           n, None) == -4
