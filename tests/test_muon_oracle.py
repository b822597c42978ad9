"""Pins of the orthogonalisation and Muon oracle (CPU): singular values, closed forms, the fp16 scheme's distance."""
import numpy as np
import pytest

from oracle import ops_oracle as oo


def _poly(s, coefficients):
    for a, b, c in coefficients:
        s = a * s + b * s ** 3 + c * s ** 5
    return s


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6), (1, 4), (4, 1)])
def test_singular_values_follow_the_polynomial(shape):
    x = np.random.default_rng(0).normal(size=shape)
    u, s, v = np.linalg.svd(x, full_matrices=False)
    k = ((3.0, -3.2, 1.2), (2.0, -1.5, 0.5), (1.5, -0.5, 0.0))
    ref = u * _poly(s / (np.linalg.norm(x) + 0.1), k) @ v
    np.testing.assert_allclose(oo.orthogonalize(x, k, 0.1), ref, rtol=1e-12, atol=1e-12)


def test_closed_forms():
    assert np.all(oo.orthogonalize(np.zeros((3, 4))) == 0)
    k = ((1.5, -0.5, 0.0),) * 40  # converges to the orthogonal factor
    q = oo.orthogonalize(np.random.default_rng(1).normal(size=(4, 7)), k)
    np.testing.assert_allclose(q @ q.T, np.eye(4), atol=1e-12)
    np.testing.assert_allclose(oo.orthogonalize([[3.0, 4.0]], k, 0.0), [[0.6, 0.8]])


def test_usual_coefficients_bring_singular_values_near_1():
    x = np.random.default_rng(2).normal(size=(60, 100))
    s = np.linalg.svd(oo.orthogonalize(x), compute_uv=False)
    assert s.min() > 0.65 and s.max() < 1.25


@pytest.mark.parametrize("kind", ["gauss", "low rank"])
def test_the_fp16_scheme_is_near(kind):
    """The bound that the kernels are held to (test_gpu_muon.py) holds for the scheme itself."""
    rng = np.random.default_rng(3)
    x = rng.normal(size=(200, 300))
    if kind == "low rank":
        x = rng.normal(size=(200, 8)) @ rng.normal(size=(8, 300)) + 0.02 * x
    ref = oo.orthogonalize(x)
    assert np.linalg.norm(oo.orthogonalize_fp16(x) - ref) <= 5e-3 * np.linalg.norm(ref)


def test_muon_step_by_hand():
    w, g, m = np.ones((1, 2)), np.array([[3.0, 4.0]]), np.zeros((1, 2))
    k = ((1.5, -0.5, 0.0),) * 40
    w1, m1 = oo.muon(w, g, m, lr=0.1, momentum=0.5, nesterov=True, weight_decay=0.2, scale=2.0, coefficients=k, eps=0.0)
    np.testing.assert_allclose(m1, [[1.5, 2.0]])
    np.testing.assert_allclose(w1, 0.98 - 0.2 * np.array([[0.6, 0.8]]))
