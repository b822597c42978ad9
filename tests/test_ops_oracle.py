"""Pins of the token log-probability and AdamW oracle (CPU): closed forms, differences, invariants."""
import numpy as np
import pytest
from scipy.special import log_softmax

from oracle import ops_oracle as oo


def test_logprobs_against_scipy_and_uniform_rows():
    rng = np.random.default_rng(0)
    z = rng.normal(size=(5, 37)) * 3
    t = rng.integers(0, 37, 5)
    lp, H, top, ids = oo.token_logprobs(z, t, 0.7, 4)
    ref = log_softmax(z / 0.7, axis=1)
    np.testing.assert_allclose(lp, ref[np.arange(5), t], rtol=1e-13)
    np.testing.assert_allclose(H, -(np.exp(ref) * ref).sum(1), rtol=1e-13)
    np.testing.assert_allclose(top, -np.sort(-ref, axis=1)[:, :4], rtol=1e-13)
    lp, H, _, ids = oo.token_logprobs(np.zeros((1, 8)), [3], 1.0, 8)
    assert lp[0] == -np.log(8) and abs(H[0] - np.log(8)) < 1e-15 and list(ids[0]) == list(range(8))


def test_masked_and_ignored_rows():
    z = np.array([[0.0, -np.inf, 1.0], [-np.inf] * 3, [0.0, 0.0, 0.0]])
    lp, H, top, ids = oo.token_logprobs(z, [1, 0, -100], 1.0, 3)
    assert lp[0] == -np.inf and lp[1] == -np.inf and lp[2] == 0
    assert H[1] == 0 and list(ids[0]) == [2, 0, 1] and list(ids[1]) == [0, 1, 2] and top[0, 2] == -np.inf
    d = oo.token_logprobs_grad(z, [2, 0, -100], 1.0, np.ones(3), np.zeros(3))
    assert np.all(d[1:] == 0) and d[0, 1] == 0 and abs(d[0].sum()) < 1e-15


@pytest.mark.parametrize("tau", [0.5, 1.0, 3.0])
def test_gradient_against_differences(tau):
    rng = np.random.default_rng(3)
    z, t = rng.normal(size=(4, 9)), np.array([0, 8, -1, 4])
    gl, ge = rng.normal(size=4), rng.normal(size=4)

    def f(x):
        lp, H, _, _ = oo.token_logprobs(x, t, tau)
        return (gl * lp + ge * H).sum()

    d = oo.token_logprobs_grad(z, t, tau, gl, ge)
    for i in np.ndindex(z.shape):
        e = np.zeros_like(z)
        e[i] = 1e-5
        assert abs((f(z + e) - f(z - e)) / 2e-5 - d[i]) < 1e-8


def test_adamw_against_torch():
    import torch
    rng = np.random.default_rng(5)
    p = torch.tensor(rng.normal(size=50), dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
    w, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.normal(size=50)
        p.grad = torch.tensor(g)
        opt.step()
        w, m, v = oo.adamw(w, g, m, v, step=step, lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.3)
        np.testing.assert_allclose(w, p.detach().numpy(), rtol=1e-13)


def test_codes_are_e4m3_values_and_unbiased():
    import torch
    rng = np.random.default_rng(6)
    x = rng.normal(size=700) * np.exp2(rng.integers(-12, 3, 700))
    total = np.zeros(700)
    reps = 400
    for s in range(reps):
        q, e = oo.round_code(x, oo.random_bits(s, 0, 700) & np.uint64(0xFFFF), False)
        assert np.array_equal(torch.tensor(q).to(torch.float8_e4m3fn).double().numpy(), q)
        total += q * np.exp2(np.repeat(e, 256)[:700])
    r, step, e = oo.code_parts(x)
    one = step * np.exp2(np.repeat(e, 256)[:700])  # one rounding is off by a Bernoulli variable of this step
    assert np.all(np.abs(total / reps - x) <= 5 * 0.5 * one / np.sqrt(reps))
    top = np.abs(np.pad(x, (0, 68))).reshape(-1, 256).max(1) * np.exp2(-e)
    assert np.all((top >= 128) & (top < 256))


def test_random_bits_of_known_positions():
    """The finaliser's published fixed point and the high half of a position."""
    assert oo.mix32(np.array([0], np.uint64))[0] == 0
    assert oo.mix32(np.array([1], np.uint64))[0] == 0x514E28B7  # MurmurHash3 x86_32 of an empty key, seed 1
    a, b = oo.random_bits(7, 2 ** 32 - 1, 2)
    assert oo.random_bits(7, 0, 1)[0] != b and a == oo.random_bits(7, 2 ** 32 - 1, 1)[0]
