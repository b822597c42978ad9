"""8-bit states: an element whose moments are not finite takes neither its block's scale nor its neighbours' states with it."""
import pytest
import torch

from hybrid_upcycling_gb300 import State8, _lib, adamw_step, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def step(param, grad, bad, at, n=5000):
    gen = torch.Generator("cuda").manual_seed(3)
    rnd = lambda s: torch.randn(n, generator=gen, device="cuda") * s  # noqa: E731
    w, g = rnd(0.02), rnd(1e-3).to(grad)
    p = [w.clone() if param == "fp32" else w.bfloat16()]
    m, v = State8.zeros_like(w), State8.zeros_like(w)
    masters = [w] if param == "master" else None
    adamw_step(p, [rnd(1e-3).to(grad)], [m], [v], step=1, lr=1e-3, masters=masters, seed=1)
    for s in (m, v):  # so that the bad element is not its block's largest without its gradient
        s.codes.view(torch.uint8)[at] = 0
    g[at] = bad
    adamw_step(p, [g], [m], [v], step=2, lr=1e-3, masters=masters, seed=2)
    return [p[0], m.codes.view(torch.uint8), v.codes.view(torch.uint8), w] if masters else \
        [p[0], m.codes.view(torch.uint8), v.codes.view(torch.uint8)], m, v


@pytest.mark.parametrize("param", ["fp32", "master", "bf16"])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30])
@pytest.mark.parametrize("at", [300, 1024, 4999])
def test_neighbours_are_those_of_a_step_without_it(param, grad, bad, at):
    good, gm, gv = step(param, grad, 0.0, at)
    now, m, v = step(param, grad, bad, at)
    others = torch.ones(5000, dtype=torch.bool, device="cuda")
    others[at] = False
    huge = bad == 1e30  # its square overflows, its first moment does not: that one is a value, and the largest of its block
    for i, (a, b) in enumerate(zip(good, now)):
        assert (huge and i == 1) or torch.equal(a[others], b[others]), i
    assert torch.equal(gv.exponents, v.exponents) and (huge or torch.equal(gm.exponents, m.exponents))
    assert torch.isnan(v.values()[at]) and torch.isnan(m.values()[at]).item() != huge
    assert torch.isfinite(v.values()[others]).all() and torch.isfinite(now[0][others].float()).all()
    assert torch.isfinite(now[0][at].float()).item() == huge
