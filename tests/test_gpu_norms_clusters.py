"""Gradients of norms whose rows a cluster of thread blocks shares, with many rows for each cluster: the exchanged sums, their three
places and the phases of their barriers are used several times over. Against the fp64 oracle, with the bounds of test_gpu_norms.py.

Clusters of a row: 152 / CTAs of a row (two CTAs an SM where they have at most 288 threads), so these cases take 5 to 20 rows each.
"""
import os
import re

import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build
from oracle import ops_oracle as oo
from test_gpu_norms import DT, U, Bounds, check, f64, make, run

SOURCE = os.path.join(build.CSRC, "norm.cu")

CASES = [  # rows, columns, type, gain's type, bias, residual, RMS
    (1501, 6000, "bf16", "same", False, True, True),     # one CTA
    (1501, 6000, "bf16", "fp32", True, False, False),
    (1201, 8200, "fp16", "same", True, True, False),     # two, two of them an SM
    (1201, 8200, "bf16", "same", False, False, True),
    (1001, 16384, "bf16", "same", True, False, False),   # two
    (1001, 16384, "bf16", "fp32", False, True, True),
    (401, 8192, "fp32", "same", True, True, False),
    (401, 8192, "fp32", "same", False, False, True),
    (601, 33000, "bf16", "fp32", True, True, False),     # five
    (601, 20000, "fp32", "same", False, True, True),
    (301, 65536, "bf16", "same", False, False, True),    # eight
    (301, 32768, "fp32", "same", True, False, False),
]


def test_sums_from_other_thread_blocks_are_acquired_at_cluster_scope():
    """What another CTA of the cluster sends with st.async it releases at cluster scope: the wait for it has to acquire at that scope."""
    waits = re.findall(r"(wait_bounded\S*)\((arrived\b)", open(SOURCE).read())
    assert waits and all(w == "wait_bounded<true>" for w, _ in waits)


@pytest.mark.gpu
@pytest.mark.parametrize("N,d,dtype,gain,bias,residual,rms", CASES)
def test_many_rows_of_a_cluster(N, d, dtype, gain, bias, residual, rms):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    dtype, eps = DT[dtype], 1e-4
    x, r, w, b, dy, ds = make(N, d, dtype, gain, bias, residual, seed=N + d)
    leaves = [t.requires_grad_() for t in (x, r, w, b) if t is not None]
    y, total = run(x, r, w, b, eps, rms)
    grads = torch.autograd.grad([y] if total is None else [y, total], leaves, [dy] if ds is None else [dy, ds])
    _lib.hylo_kl_sync_status()
    grads = dict(zip([n for n, t in zip("xrwb", (x, r, w, b)) if t is not None], grads))
    s = f64(x if total is None else total)
    bounds = Bounds(s, f64(w), f64(b), eps, rms)
    check(y, bounds.y, bounds.dy, dtype, "y")
    rdx, rdw, rdb = oo.norm_grad(s, f64(w), eps, rms, f64(dy))
    bdx, bdw, bdb = bounds.grads(f64(dy))
    if residual:
        rdx = rdx + f64(ds)
        bdx = bdx + U * abs(rdx)
    check(grads["x"], rdx, bdx, dtype, "dx")
    check(grads["w"], rdw, bdw, w.dtype, "dw")
    if bias:
        check(grads["b"], rdb, bdb, b.dtype, "db")
