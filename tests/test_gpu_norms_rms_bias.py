"""RMS norm with a bias, which the C entry points offer (rms_norm of the package has none): every kernel of the forward and of the
backward against the fp64 oracle, with the bounds of test_gpu_norms.py."""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build
from oracle import ops_oracle as oo
from test_gpu_norms import DT, U, Bounds, check, f64, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


@pytest.mark.parametrize("dtype,gain,residual", [("bf16", "same", True), ("bf16", None, False), ("fp32", "same", False), ("fp16", "fp32", True)])
@pytest.mark.parametrize("N,d,pad", [
    (3, 2048, 0), (5, 40, 0), (2, 8192, 0),      # few rows
    (3, 255, 1),                                 # few odd rows
    (2001, 2048, 0), (5001, 96, 0),              # whole vectors, many rows
    (801, 6000, 0), (9, 9000, 8), (9, 12288, 0), (700, 8192, 0),  # and wider ones
    (801, 1001, 0), (301, 5001, 3), (9, 9001, 0),  # odd rows
    (5, 20000, 0), (3, 70000, 0),                # read several times
])
def test_rms_norm_with_a_bias(N, d, pad, dtype, gain, residual):
    dtype, eps = DT[dtype], 1e-4
    x, r, w, b, dy, ds = make(N, d, dtype, gain or "same", True, residual, pad, seed=N + d)
    if gain is None:  # a bias alone
        w = None
    total = torch.empty(N, d, dtype=dtype, device="cuda") if residual else None
    y = torch.empty(N, d, dtype=dtype, device="cuda")
    stats = torch.empty(N, 2, device="cuda")
    _lib.hylo_norm(x, r, w, b, True, eps, total, y, stats)
    s = f64(total if residual else x)
    bounds = Bounds(s, f64(w), f64(b), eps, True)
    check(y, bounds.y, bounds.dy, dtype, "y")
    assert torch.count_nonzero(stats[:, 0]) == 0
    dx = torch.empty_like(y)
    dw, db = (torch.empty_like(b) for _ in range(2))
    ws = torch.empty(_lib.hylo_norm_backward_workspace_bytes(N, d), dtype=torch.uint8, device="cuda")
    _lib.hylo_norm_backward(total if residual else x, w, True, stats, dy, ds, dx, dw, db, ws)
    _lib.hylo_kl_sync_status()
    rdx, rdw, rdb = oo.norm_grad(s, f64(w), eps, True, f64(dy))
    bdx, bdw, bdb = bounds.grads(f64(dy))
    if residual:
        rdx = rdx + f64(ds)
        bdx = bdx + U * abs(rdx)
    check(dx, rdx, bdx, dtype, "dx")
    check(dw, rdw, bdw, b.dtype, "dw")
    check(db, rdb, bdb, b.dtype, "db")
