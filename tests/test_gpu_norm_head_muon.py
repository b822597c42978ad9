"""Norms, the LM head's loss and Muon as a training step uses them together: gradients through all of them, a step, the example.

Tolerance of the gradients. Everything between two operators is bf16: a rounding is off by at most 2^-8 of a value, so of a
tensor's norm too, and by 2^-8 / sqrt(12) = 1.1e-3 of it in the root mean square over values and binades (at most 2^-8 /
sqrt(3) = 2.3e-3). A gradient of this model has passed at most 3 roundings a layer forwards (norm, product, sum), 4 backwards
(dx, the two products, the sum of two streams), and the head's gradient two more: with two layers 2 x 7 + 4 = 18 of them. What a
step passes on is not larger than what it got, but for norms (by 1 / r, which the next norm takes back) and sums of
streams (by 2 where both agree), so independent roundings give 2 x 2.3e-3 sqrt(18) = 2.0e-2 of the norm.
"""
import importlib.util
import os

import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import AdamW, Muon, build, head_logprobs
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
TOL = 2e-2


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def leaves(tokens, d, V, layers, seed=0):
    gen = torch.Generator("cuda").manual_seed(seed)

    def rand(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std + mean).bfloat16().requires_grad_()

    h, W = rand(tokens, d), rand(V, d, std=0.1)
    gains = [rand(d, std=0.1, mean=1.0) for _ in range(layers + 1)]
    mats = [rand(d, d, std=d ** -0.5) for _ in range(layers)]
    target = torch.randint(0, V, (tokens,), generator=gen, device="cuda")
    target[::5] = -1
    return h, W, gains, mats, target


def plain(h, W, gains, mats, target):
    """The loss from the definitions, in the type of its arguments."""
    def norm(x, w):
        return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w

    s, y = h, norm(h, gains[0])
    for P, w in zip(mats, gains[1:]):
        s = s + y @ P.t()
        y = norm(s, w)
    logp = (y @ W.t()).log_softmax(-1)
    keep = (target >= 0).nonzero().squeeze(1)
    return -logp[keep, target[keep]].sum() - 0.3 * -(logp.exp() * logp).sum()


def fused(ex, h, W, gains, mats, target):
    logp, entropy = head_logprobs(ex.student(h, gains, mats), W, target)
    return -logp.sum() - 0.3 * entropy.sum()


def grads(loss, h, W, gains, mats):
    return torch.autograd.grad(loss, [h, W, *gains, *mats])


@pytest.mark.parametrize("tokens,d,V,layers", [(1, 64, 50, 1), (37, 136, 301, 2), (300, 256, 1000, 2)])
def test_gradients_through_norms_and_head(ex, tokens, d, V, layers):
    h, W, gains, mats, target = leaves(tokens, d, V, layers, tokens)
    got = grads(fused(ex, h, W, gains, mats, target), h, W, gains, mats)
    x = [[t.detach().double().cpu().requires_grad_() for t in part] for part in ([h, W], gains, mats)]
    (h6, W6), gains6, mats6 = x
    want = grads(plain(h6, W6, gains6, mats6, target.cpu()), h6, W6, gains6, mats6)
    for a, b in zip(got, want):
        err = (a.double().cpu() - b).norm() / b.norm()
        assert err <= TOL, (tuple(b.shape), err.item())


def test_gradients_against_differences(ex):
    """The 64-bit loss along one direction of each leaf, against the kernels' gradients: the differences' own error is below
    1e-6, so the tolerance is that of the gradients times the direction's part of them (a direction near the gradient)."""
    h, W, gains, mats, target = leaves(50, 128, 200, 2, 4)
    params = [h, W, *gains, *mats]
    got = grads(fused(ex, h, W, gains, mats, target), h, W, gains, mats)
    x = [p.detach().double().cpu() for p in params]

    def loss(values):
        return plain(values[0], values[1], values[2:5], values[5:], target.cpu()).item()

    for i, g in enumerate(got):
        v = g.double().cpu() / g.double().norm().item()
        step = 1e-5 * x[i].norm().item()
        ends = [loss(x[:i] + [x[i] + k * step * v] + x[i + 1:]) for k in (-1, 1)]
        slope = (ends[1] - ends[0]) / (2 * step)
        norm = g.double().norm().item()
        assert abs(slope - norm) <= TOL * norm, (i, slope, norm)


@pytest.mark.parametrize("masters", [False, True])
def test_a_step_of_both_optimisers(ex, masters):
    """Three steps of a residual model: what Muon does with the gradients that came through the norms, against the oracle's
    step from the same gradients and momenta; AdamW steps the rest, and the next forward sees both."""
    h, W, gains, mats, target = leaves(64, 128, 300, 2, 5)
    muon = Muon(mats, lr=0.02, weight_decay=0.1, masters=masters, adjust="rms", seed=3)
    adamw = AdamW([h, W, *gains], lr=1e-3, masters=masters, max_norm=1.0)
    scale = 0.2 * 128 ** 0.5
    for _ in range(3):
        before = [t.detach().clone() for t in (muon.masters or mats)]
        momenta = [m.clone() for m in muon.momenta]
        for p in (h, W, *gains, *mats):
            p.grad = None
        fused(ex, h, W, gains, mats, target).backward()
        # With masters these move: a step of 1e-3 is less than half of bf16's step of 2^-7 at a gain near 1.
        stepped = adamw.masters if masters else [h, W, *gains]
        old = [t.detach().clone() for t in stepped]
        muon.step()
        adamw.step()
        assert all(not torch.equal(a, b) for a, b in zip(old, stepped))
        for i, P in enumerate(mats):
            w, m = oo.muon(*(t.double().cpu().numpy() for t in (before[i], P.grad, momenta[i])), lr=0.02, momentum=0.95, nesterov=True,
                           weight_decay=0.1, scale=scale)
            move = 0.02 * scale * 128 ** 0.5 * 1.2  # of the parameter, in the Frobenius norm: singular values up to 1.2
            now = (muon.masters or mats)[i].detach().double().cpu().numpy()
            err = np.linalg.norm(now - w)
            # 5e-3 of the update's norm; without masters one stochastic rounding, up to a whole step of 2^-7
            assert err <= 5e-3 * move + (2.0 ** -24 if masters else 2.0 ** -7) * np.linalg.norm(w), err
            assert np.abs(muon.momenta[i].double().cpu().numpy() - m).max() <= 3 * 2.0 ** -24 * np.abs(m).max()
            if masters:
                assert torch.equal(P.detach(), muon.masters[i].bfloat16())
    assert torch.isfinite(fused(ex, h, W, gains, mats, target))


def test_forward_of_the_layers_in_a_graph(ex):
    """Norms and head without gradients, captured once and replayed on new hidden states: what the eager calls give."""
    h, W, gains, mats, target = leaves(40, 128, 300, 2, 6)
    h = h.detach()
    with torch.no_grad():
        first = head_logprobs(ex.student(h, gains, mats), W, target)[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = head_logprobs(ex.student(h, gains, mats), W, target)[0]
        graph.replay()
        assert torch.equal(out, first)
        h.copy_(torch.randn_like(h))
        graph.replay()
        assert torch.equal(out, head_logprobs(ex.student(h, gains, mats), W, target)[0])


@pytest.mark.parametrize("bits,masters", [(8, False), (32, True)])
def test_the_example_runs_with_layers(ex, bits, masters):
    losses, before, after, top = ex.train(steps=3, tokens=300, hidden=64, vocab=1000, state_bits=bits, masters=masters, layers=2)
    assert len(losses) == 3 and all(np.isfinite([*losses, before, after]))
    assert top.top_tokens.shape == (4, 5)
