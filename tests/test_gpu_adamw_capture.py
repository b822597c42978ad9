"""An AdamW step is refused while its stream is being captured: a replay would repeat the captured step number, learning
rate and random bits. The gradient norm can be captured."""
import pytest
import torch

from hybrid_upcycling_gb300 import AdamW, _lib, adamw_step, build, grad_norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_is_refused_and_changes_nothing(bits):
    p = torch.ones(3000, device="cuda", requires_grad=True)
    g = torch.full((3000,), 0.5, device="cuda")
    opt = AdamW([p], lr=0.1, weight_decay=0.0, state_bits=bits, max_norm=1e6)
    opt.step([g])
    torch.cuda.synchronize()
    keep, x, graph = p.detach().clone(), torch.zeros(3, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x += 1
        with pytest.raises(_lib.HyloError) as e:
            opt.step([g])
        assert e.value.status == -9 and "captured" in str(e.value)
    for _ in range(3):
        graph.replay()
    assert opt.steps == 1 and torch.equal(p, keep) and torch.all(x == 3)  # what else was captured still replays
    opt.step([g])
    assert opt.steps == 2 and torch.all(p < keep)


def test_a_captured_norm_replays_on_new_gradients():
    g = [torch.randn(70000, device="cuda"), torch.randn(33, device="cuda")]
    grad_norm(g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = grad_norm(g)
    for _ in range(3):
        for x in g:
            x.normal_()
        graph.replay()
        assert torch.equal(norm, grad_norm(g))


def test_another_streams_capture_does_not_refuse():
    """Capture is a property of the stream: a step on a stream that is not captured runs."""
    p, g, m, v = (torch.ones(100, device="cuda") for _ in range(4))
    side, graph, x = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.zeros(3, device="cuda")
    adamw_step([p], [g], [m], [v], step=1, lr=0.1)
    torch.cuda.synchronize()
    keep = p.clone()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        x += 1
        with torch.cuda.stream(side):
            adamw_step([p], [g], [m], [v], step=2, lr=0.1)
    torch.cuda.synchronize()
    assert torch.all(p < keep)
