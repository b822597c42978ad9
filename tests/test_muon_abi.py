"""Refusals of orthogonalize and muon_step: the C entry points with bad arguments (these calls never reach the GPU) and
the checks of the Python functions."""
import ctypes
import struct

import pytest
import torch

from hybrid_upcycling_gb300 import Muon, _lib, build, muon_step, orthogonalize

X, Y, P, G, W, M, WS = (0x1000000 * (1 + i) for i in range(7))
BIG = 1 << 60


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _orth(lib, mats=None, count=None, dt=0, odt=1, steps=1, k=(3.4, -4.7, 2.0), eps=1e-7, ws=1 << 40, nbytes=1 << 30, **kw):
    row = dict(x=X, out=Y, rows=20, cols=30, ld=30)
    row.update(kw)
    rows = [row] if mats is None else [{**row, **m} for m in mats]
    table = b"".join(struct.pack("=" + _lib.ORTH_MATRIX, *r.values()) for r in rows)
    c = None if k is None else (ctypes.c_double * len(k))(*k)
    return lib.hylo_orthogonalize(table, len(rows) if count is None else count, dt, odt, steps, c, eps, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), -1), (dict(out=0), -1), (dict(ws=None), -1), (dict(k=None), -1), (dict(count=-1), -2), (dict(rows=-1), -2),
    (dict(cols=(1 << 20) + 1), -2), (dict(rows=16385, cols=16385, ld=16385), -2), (dict(ld=29), -2), (dict(dt=3), -2), (dict(odt=0), -2),
    (dict(steps=0), -2), (dict(steps=33), -2), (dict(x=X + 2), -3), (dict(out=Y + 1), -3), (dict(ws=(1 << 40) + 16), -3),
    (dict(eps=-1.0), -4), (dict(eps=float("nan")), -4), (dict(k=(float("inf"), 0.0, 0.0)), -4), (dict(k=(1e7, 0.0, 0.0)), -4),
    (dict(k=(2.0,) * 96, steps=32), -4), (dict(nbytes=1000), -5), (dict(out=X + 64), -2), (dict(mats=[dict(), dict(x=X + (1 << 22))]), -2),
    (dict(ws=X - 256), -2), (dict(mats=[dict(), dict(out=Y + 600, x=X + (1 << 22))]), -2),
])
def test_orthogonalize_refuses(lib, kw, status):
    assert _orth(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def _muon(lib, tensors=None, pdt=1, gdt=0, mu=0.9, steps=1, k=(3.4, -4.7, 2.0), eps=1e-7, scale=1.0, norm=None, max_norm=1.0, ws=1 << 40,
          nbytes=1 << 30, **kw):
    t = dict(p=P, g=G, w=W, m=M, rows=20, cols=30, lr=1e-3, wd=0.1, s=1.0)
    t.update(kw)
    rows = [t] if tensors is None else [{**t, **x} for x in tensors]
    table = b"".join(struct.pack("=" + _lib.MUON_TENSOR, *r.values()) for r in rows)
    return lib.hylo_muon_step(table, len(rows), pdt, gdt, mu, 1, steps, (ctypes.c_double * 3)(*k), eps, scale, norm, max_norm, 0, ws, nbytes,
                              None)


@pytest.mark.parametrize("kw,status", [
    (dict(p=0), -1), (dict(g=0), -1), (dict(m=0), -1), (dict(ws=None), -1), (dict(pdt=2), -2), (dict(gdt=2), -2), (dict(mu=1.0), -2),
    (dict(mu=-0.1), -2), (dict(mu=float("nan")), -2), (dict(pdt=0), -2), (dict(tensors=[dict(), dict(w=0, p=P + 4096, g=G + 4096, m=M + 4096)]), -2),
    (dict(rows=1 << 21), -2), (dict(p=P + 1), -3), (dict(w=W + 2), -3), (dict(m=M + 1), -3), (dict(norm=0x10000002), -3),
    (dict(lr=float("inf")), -4), (dict(wd=float("nan")), -4), (dict(s=float("inf")), -4), (dict(scale=float("nan")), -4),
    (dict(norm=0x10000000, max_norm=0.0), -4), (dict(nbytes=4096), -5), (dict(m=G), -2), (dict(w=P), -2), (dict(tensors=[dict(), dict()]), -2),
    (dict(norm=M + 8), -2), (dict(eps=-1.0), -4),
])
def test_muon_refuses(lib, kw, status):
    assert _muon(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def test_workspace(lib):
    def q(*shapes):
        table = b"".join(struct.pack("=" + _lib.ORTH_MATRIX, X, Y, r, c, c) for r, c in shapes)
        assert lib.hylo_orthogonalize_workspace_bytes(table, len(shapes)) == \
            lib.hylo_muon_workspace_bytes(b"".join(struct.pack("=" + _lib.MUON_TENSOR, P, G, W, M, r, c, 0, 0, 1) for r, c in shapes), len(shapes))
        return lib.hylo_orthogonalize_workspace_bytes(table, len(shapes))

    square, ctrl, part = 5 * 256 * 256 * 2, 512, 256 * 1024  # X twice, its second term, A, B; the work's counters; one part of a tile's sum
    assert q((200, 200)) == square + 256 + ctrl and q((200, 200), (0, 5)) == square + 256 + ctrl
    assert q((1, 1), (256, 256)) == 2 * square + 256 + ctrl
    # 36 tiles leave room for two parts of their sums each, one tile for as many as are worth while
    assert q((2048, 8192)) == q((8192, 2048)) == 3 * 2048 * 8192 * 2 + 2 * 2048 * 2048 * 2 + 1024 * 12 + 2816 + 36 * 2 * part
    assert q(*[(2048, 8192)] * 100) <= 1025 << 20 and q(*[(64, 64)] * 1000) == 64 * square + 64 * 12 + ctrl
    assert q((200, 8193)) == 256 * (3 * 8448 + 2 * 256) * 2 + 256 * 10 + ctrl + 4 * part
    assert q((100, 1 << 20)) == 256 * (3 * (1 << 20) + 2 * 256) * 2 + 1024 * 12 + ctrl + 50 * part + 256 * 128 * 1024  # deep parts
    assert q((0, 0)) == ctrl and q((1 << 21, 1)) == 0


def test_table_layouts_are_the_headers():
    assert struct.calcsize("=" + _lib.ORTH_MATRIX) == 40 and struct.calcsize("=" + _lib.MUON_TENSOR) == 72


def test_python_checks():
    x, v = torch.zeros(6, 8), torch.zeros(8)
    for bad in (lambda: orthogonalize([x]), lambda: orthogonalize(x),  # not on a GPU
                lambda: orthogonalize(v), lambda: orthogonalize(x.double()), lambda: orthogonalize([x, x.bfloat16()]),
                lambda: orthogonalize(x, dtype=torch.float32), lambda: orthogonalize(x, coefficients=(1.0, 2.0)),
                lambda: orthogonalize(x, steps=3, coefficients=[(1.0, 0.0, 0.0)] * 2),
                lambda: muon_step([x], [x], [x], lr=0.1), lambda: muon_step([x], [x], [], lr=0.1),
                lambda: muon_step([x], [x], [x], lr=0.1, adjust="other"), lambda: Muon([]), lambda: Muon([v]), lambda: Muon([x, x]),
                lambda: Muon([x, x.bfloat16()]), lambda: Muon([{"params": [x], "momentum": 0.5}]), lambda: Muon([x], adjust="big")):
        with pytest.raises(ValueError):
            bad()
