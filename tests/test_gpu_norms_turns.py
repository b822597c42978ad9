"""Norms of many rows against the fp64 oracle, element by element: a thread block with a ring in shared memory takes 5 to 20 turns, so
that the ring goes round and column sums run over many rows; one that reads its rows several times takes up to 5. Bounds are those
of test_gpu_norms.py. (Rows that a cluster shares are in test_gpu_norms_clusters.py.)

The numbers of rows are such that the last turn is not whole, and taken from the grids: at most 152 x 512 / threads of a row thread
blocks (forward of up to 4096 columns: 152 x 768), with 128 / threads rows where these are 32 or fewer, two at a time in 16 bits.
"""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build
from oracle import ops_oracle as oo
from test_gpu_norms import DT, U, Bounds, check, f64, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


CASES = [  # rows, columns, type, gain's type, bias, residual, row padding, RMS
    # whole vectors, several rows a thread block
    (80_021, 72, "fp16", "fp32", True, True, 0, False),
    (80_021, 72, "bf16", "same", False, False, 8, True),
    (40_009, 200, "bf16", "fp32", True, False, 0, False),
    (40_009, 132, "fp32", "same", False, True, 4, True),
    # one
    (6011, 2048, "bf16", "same", True, True, 0, False),
    (6011, 2048, "bf16", "fp32", False, True, 8, True),
    (6011, 2048, "fp32", "same", True, True, 0, False),
    (6011, 2048, "fp32", None, False, False, 0, True),
    (3001, 4096, "fp16", "same", True, False, 0, False),
    # 16 and 32 columns a thread in the forward
    (1501, 8192, "bf16", "same", True, True, 0, False),
    (1009, 12_288, "bf16", "same", False, True, 0, True),
    (1009, 16_384, "fp32", "same", True, False, 0, False),
    # odd rows: part of a warp, whole warps, wider ones
    (100_003, 31, "fp32", "same", True, True, 0, False),
    (100_003, 45, "bf16", "fp32", False, True, 1, True),
    (9001, 1001, "bf16", "same", True, True, 0, False),
    (9001, 1001, "fp16", "fp32", False, False, 23, True),
    (9001, 1001, "fp32", "same", True, False, 0, False),
    (2003, 5001, "bf16", "same", True, True, 3, False),
    (2003, 5001, "fp32", "same", False, True, 0, True),
    (1009, 9001, "bf16", "fp32", True, True, 0, False),
    # rows that are read several times
    (1501, 20_000, "bf16", "same", True, True, 0, False),
    (1301, 10_000, "fp32", "same", True, True, 0, False),
    (351, 70_000, "bf16", "fp32", False, True, 0, True),
    (701, 33_001, "fp32", "same", True, False, 0, False),
]


@pytest.mark.parametrize("N,d,dtype,gain,bias,residual,pad,rms", CASES)
def test_many_rows_of_a_thread_block(N, d, dtype, gain, bias, residual, pad, rms):
    dtype, eps = DT[dtype], 1e-4
    x, r, w, b, dy, ds = make(N, d, dtype, gain, bias, residual, pad, seed=N + d)
    names = [n for n, t in zip("xrwb", (x, r, w, b)) if t is not None]
    leaves = [t.requires_grad_() for t in (x, r, w, b) if t is not None]
    y, total = run(x, r, w, b, eps, rms)
    grads = dict(zip(names, torch.autograd.grad([y] if total is None else [y, total], leaves, [dy] if ds is None else [dy, ds])))
    _lib.hylo_kl_sync_status()
    s = f64(x if total is None else total)
    if residual:
        assert torch.equal(total, (x.float() + r.float()).to(dtype))
        assert torch.equal(grads["x"], grads["r"])
    bounds = Bounds(s, f64(w), f64(b), eps, rms)
    check(y, bounds.y, bounds.dy, dtype, "y")
    rdx, rdw, rdb = oo.norm_grad(s, f64(w), eps, rms, f64(dy))
    bdx, bdw, bdb = bounds.grads(f64(dy))
    if residual:
        rdx = rdx + f64(ds)
        bdx = bdx + U * abs(rdx)
    check(grads["x"], rdx, bdx, dtype, "dx")
    if w is not None:
        check(grads["w"], rdw, bdw, w.dtype, "dw")
    if b is not None:
        check(grads["b"], rdb, bdb, b.dtype, "db")
