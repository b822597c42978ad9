"""Pins of the norm oracle (CPU): torch's layer norm in 64 bits, closed forms, differences."""
import numpy as np
import pytest
import torch

from oracle import ops_oracle as oo


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gain", [False, True])
def test_against_torch_in_64_bits(rms, gain):
    rng = np.random.default_rng(1)
    s, dy = rng.normal(size=(5, 12)) + 2, rng.normal(size=(5, 12))
    w, b = (rng.normal(size=12), None if rms else rng.normal(size=12)) if gain else (None, None)
    t = lambda x: None if x is None else torch.tensor(x, requires_grad=True)  # noqa: E731
    ts, tw, tb = t(s), t(w), t(b)
    f = torch.nn.functional
    y = f.rms_norm(ts, (12,), tw, 1e-4) if rms else f.layer_norm(ts, (12,), tw, tb, 1e-4)
    y.backward(torch.tensor(dy))
    ref, _, _ = oo.norm(s, w, b, 1e-4, rms)
    ds, dw, db = oo.norm_grad(s, w, 1e-4, rms, dy)
    np.testing.assert_allclose(ref, y.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(ds, ts.grad.numpy(), rtol=1e-11, atol=1e-12)
    if gain:
        np.testing.assert_allclose(dw, tw.grad.numpy(), rtol=1e-12)
        if not rms:
            np.testing.assert_allclose(db, tb.grad.numpy(), rtol=1e-12)


def test_closed_forms():
    y, mu, r = oo.norm([[1.0, 3.0]], None, None, 0.0, False)
    np.testing.assert_allclose(y, [[-1.0, 1.0]])
    assert mu[0, 0] == 2 and r[0, 0] == 1
    y, _, _ = oo.norm([[3.0, 4.0]], np.array([2.0, 1.0]), None, 0.0, True)
    np.testing.assert_allclose(y, np.array([[6.0, 4.0]]) / np.sqrt(12.5))


@pytest.mark.parametrize("rms", [False, True])
def test_gradient_against_differences(rms):
    rng = np.random.default_rng(2)
    s, dy, w = rng.normal(size=(3, 7)), rng.normal(size=(3, 7)), rng.normal(size=7)
    ds, dw, _ = oo.norm_grad(s, w, 1e-3, rms, dy)
    f = lambda a, b: (oo.norm(a, b, None, 1e-3, rms)[0] * dy).sum()  # noqa: E731
    for i in np.ndindex(s.shape):
        e = np.zeros_like(s)
        e[i] = 1e-6
        assert abs((f(s + e, w) - f(s - e, w)) / 2e-6 - ds[i]) < 1e-8
    for j in range(7):
        e = np.zeros(7)
        e[j] = 1e-6
        assert abs((f(s, w + e) - f(s, w - e)) / 2e-6 - dw[j]) < 1e-8
