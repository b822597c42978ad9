"""Arrays that an AdamW step writes may not overlap others: the thread blocks that share elements would race. The calls here are
refused before they reach the GPU."""
import struct

import pytest
import torch

from hybrid_upcycling_gb300 import AdamW, State8, _lib, adamw_step, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def rows(k, bits):
    """Addresses of k tensors, all arrays apart."""
    out = []
    for i in range(k):
        a = {x: 0x100000 + (7 * i + j) * 0x10000 for j, x in enumerate(("p", "g", "w", "m", "v", "me", "ve"))}
        a["w"] = 0
        if bits == 32:
            a["me"] = a["ve"] = 0
        out.append(a)
    return out


def call(lib, tensors, n, bits):
    table = b"".join(struct.pack("=" + _lib.ADAMW_TENSOR, *t.values(), n, 1e-3, 0.1) for t in tensors)
    return lib.hylo_adamw_step(table, len(tensors), 0, 0, bits, 0.9, 0.999, 1e-8, 1, 1.0, None, 1.0, 0, None)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("first,second,shift", [
    ((0, "p"), (1, "p"), 0), ((0, "p"), (0, "g"), 0), ((2, "m"), (0, "v"), 0), ((0, "p"), (2, "g"), 4), ((1, "g"), (2, "m"), 396),
    ((0, "m"), (0, "p"), -96)])
def test_overlaps_are_refused(lib, bits, first, second, shift):
    n = 400 if bits == 8 else 100
    t = rows(3, bits)
    t[second[0]][second[1]] = t[first[0]][first[1]] + shift
    assert call(lib, t, n, bits) == -2
    assert b"overlap" in lib.hylo_kl_last_error()


def test_overlapping_exponents_are_refused(lib):
    t = rows(2, 8)  # three exponents each
    t[1]["me"] = t[0]["ve"] + 2
    assert call(lib, t, 600, 8) == -2 and b"overlap" in lib.hylo_kl_last_error()


def test_a_parameter_given_twice_to_the_class():
    a, b = torch.zeros(4), torch.zeros(4)
    with pytest.raises(ValueError, match="twice"):
        AdamW([{"params": [a, b]}, {"params": [a]}])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_and_shared_gradients_are_not_overlaps(lib, bits):
    """Slices of one buffer that touch, and one gradient for two tensors."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    n = 300
    buf, grad = torch.randn(3 * n, device="cuda"), torch.randn(n, device="cuda")
    whole = buf.clone()
    mk = lambda k: State8.zeros_like(torch.empty(k, device="cuda")) if bits == 8 else torch.zeros(k, device="cuda")  # noqa: E731
    p = list(buf.split(n))
    adamw_step(p, [grad] * 3, [mk(n) for _ in p], [mk(n) for _ in p], step=1, lr=0.1)
    for i in range(3):
        q = [whole[i * n:(i + 1) * n].clone()]
        adamw_step(q, [grad], [mk(n)], [mk(n)], step=1, lr=0.1)
        assert torch.equal(q[0], p[i])
    for bad in ([p[0], p[0], p[1]], [buf[:n], buf[n - 1:2 * n - 1], p[2]]):
        with pytest.raises(_lib.HyloError, match="overlap"):
            adamw_step(bad, [grad] * 3, [mk(n) for _ in p], [mk(n) for _ in p], step=1, lr=0.1)
    with pytest.raises(_lib.HyloError, match="overlap"):
        adamw_step(p, p, [mk(n) for _ in p], [mk(n) for _ in p], step=1, lr=0.1)
