"""Muon steps of large matrices and long lists: whole tiles of many matrices, split sums, sums longer than the tensor cores take at a time,
several groups of matrices, in every form of the parameters.

Tolerances are those of test_gpu_muon.py. Without momentum the update is the gradient, so O is what orthogonalize gives for the same
list, and every element of a step has a few fp32 roundings, of the given random bits where a bf16 parameter has no master.
"""
import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, muon_step, orthogonalize
from oracle import ops_oracle as oo
from test_gpu_muon import EXACT, SCHEME, U, f64, matrix, rounded_up, state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


LISTS = {
    "whole tiles": [(2048, 2048)] * 3 + [(1030, 2100), (2100, 1030), (2048, 4096)],
    "split sums": [(300, 9000), (9000, 300)],
    "long split sums": [(64, 300_000)],
    "long sums": [(600, 8300)] * 8 + [(8300, 600)] * 8,          # 96 tiles: not split
    "many": [(10 + i % 7, 20 + i % 11) for i in range(150)],      # three groups of at most 64
}


@pytest.mark.parametrize("param", ["fp32", "master", "bf16"])
@pytest.mark.parametrize("name", list(LISTS))
def test_step_without_momentum_to_the_last_bit(name, param):
    p, masters, g, m = state(LISTS[name], param, "fp32")
    old = [t.clone() for t in (masters or [x.float() for x in p])]
    os = orthogonalize(g, dtype=torch.float16)
    muon_step(p, g, m, lr=0.5, momentum=0.0, weight_decay=0.1, adjust=None, masters=masters, seed=11)
    _lib.hylo_kl_sync_status()
    check_steps(p, masters, old, os, range(len(p)))
    assert all(torch.equal(a, b) for a, b in zip(m, g))


def check_steps(p, masters, old, os, which):
    starts = np.cumsum([0] + [-(-t.numel() // 256) * 256 for t in p])  # every matrix starts at a multiple of 256
    for i in which:
        o = 0.5 * os[i].double()
        ref = old[i].double() * float(np.float32(1 - 0.05)) - o
        # the returned O is rounded to fp16's subnormal numbers, half a step of which is 2^-25; the step's O is scaled
        tol = 2 * U * (ref.abs() + o.abs()) + 0.5 * 2.0 ** -25
        if masters is not None or p[i].dtype == torch.float32:
            now = (masters or p)[i]
            assert ((now.double() - ref).abs() <= tol).all(), i
            if masters is not None:
                assert torch.equal(p[i], now.bfloat16()), i
        else:  # rounding with given random bits is monotone
            bits = oo.random_bits(11, int(starts[i]), ref.numel()).reshape(ref.shape)
            bits = ((bits * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)
            lo, hi = (rounded_up((ref + s * tol).float().cpu().numpy(), bits) for s in (-1, 1))
            got = p[i].float().cpu().numpy()
            assert np.all((lo <= got) & (got <= hi)), i


def test_random_bits_of_a_second_group_by_memory():
    """24 matrices of 52 MiB of workspace each, more than a group's 1 GiB: those of the second group have their own random bits."""
    p, _, g, m = state([(1024, 8192)] * 24, "bf16", "fp32")
    old = [t.float() for t in p]
    os = orthogonalize(g, dtype=torch.float16)
    muon_step(p, g, m, lr=0.5, momentum=0.0, weight_decay=0.1, adjust=None, seed=11)
    check_steps(p, None, old, os, (0, 18, 19, 20, 23))


@pytest.mark.parametrize("param,grad", [("fp32", "fp32"), ("master", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("nesterov", [True, False])
def test_step(param, grad, nesterov):
    """Against the oracle: momentum to fp32 roundings, parameters to the orthogonalised update's accuracy (bf16 alone a whole step of
    2^-7 besides)."""
    shapes = [(1030, 2100), (2100, 1030), (300, 9000), (2, 700, 520)]
    p, masters, g, m = state(shapes, param, grad)
    w0, g0, m0 = ([f64(t) for t in ts] for ts in (masters or p, g, m))
    muon_step(p, g, m, lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, adjust="rms", masters=masters, seed=3)
    _lib.hylo_kl_sync_status()
    for i, s in enumerate(shapes):
        scale = 0.2 * np.sqrt(max(s[-2:]))
        for b in np.ndindex(s[:-2]):
            w, gg, mm = w0[i][b], g0[i][b], m0[i][b]
            rw, rm = oo.muon(w, gg, mm, lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, scale=scale)
            assert np.all(np.abs(f64(m[i])[b] - rm) <= 4 * U * (np.abs(mm) + np.abs(gg)))
            tol = (EXACT + 2.0 ** -11) * np.linalg.norm(w * (1 - 0.02 * 0.1) - rw) + 4 * U * np.linalg.norm(w)
            err = np.linalg.norm(f64((masters or p)[i])[b] - rw)
            assert err <= tol + (2.0 ** -7 * np.linalg.norm(rw) if param == "bf16" else 0), (s, err, tol)
        if masters is not None:
            assert torch.equal(p[i], masters[i].bfloat16())


def test_long_sums_of_every_product():
    """A short side of more than 8192: the sums of all three products leave the tensor cores in between. One step, in 64 bits by torch."""
    x = matrix(8300, 8400, 1)
    y = orthogonalize(x, steps=1, dtype=torch.float16).double()
    _lib.hylo_kl_sync_status()
    z = x.double()
    z /= z.norm() + 1e-7
    a, b, c = oo.MUON
    gram = z @ z.T
    want = a * z + (b * gram + c * (gram @ gram)) @ z
    h = torch.finfo(torch.float16).eps / 2
    assert ((y - want).norm() <= (EXACT + h) * want.norm() + 2.0 ** -25 * want.numel() ** 0.5).item()


def test_whole_tiles_against_the_scheme():
    """One step of a 2048 x 2048 matrix against the oracle that rounds where the kernels round."""
    x = matrix(2048, 2048, 7, "low")
    y = orthogonalize(x, steps=1, dtype=torch.float16)
    want = oo.orthogonalize_fp16(f64(x), (oo.MUON,))
    assert np.linalg.norm(f64(y) - want) <= (SCHEME + 2.0 ** -11) * np.linalg.norm(want) + 2.0 ** -25 * 2048
