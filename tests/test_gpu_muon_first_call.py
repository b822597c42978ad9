"""orthogonalize captured into a CUDA graph before any eager call of it, as the C header allows once some call has run: its kernels are
set up during the capture."""
import subprocess
import sys

import pytest
import torch

from hybrid_upcycling_gb300 import build

pytestmark = pytest.mark.gpu

CODE = """
import torch
from hybrid_upcycling_gb300 import orthogonalize, rms_norm
rms_norm(torch.ones(2, 64, device="cuda"))
x = torch.randn(300, 200, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = orthogonalize(x)
for _ in range(2):
    graph.replay()
    assert torch.equal(y, orthogonalize(x))
    x.normal_()
"""


def test_the_first_call_may_be_captured():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    r = subprocess.run([sys.executable, "-c", CODE], cwd=build.ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
