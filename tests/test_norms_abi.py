"""Refusals of the norms: the C entry points with bad arguments (these calls never reach the GPU) and the checks of the
Python functions."""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, layer_norm, rms_norm

X, R, S, Y, W, B, ST, DY, DS, DX, DW, DB, WS = (0x10000 * (1 + i) for i in range(13))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _fwd(lib, **kw):
    a = dict(x=X, r=R, dt=1, N=4, d=100, ldx=100, ldr=100, w=W, b=B, gdt=0, rms=0, eps=1e-5, s=S, y=Y, st=ST)
    a.update(kw)
    return lib.hylo_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), -1), (dict(y=None), -1), (dict(r=None), -1), (dict(s=None), -1), (dict(dt=3), -2), (dict(gdt=2), -2),
    (dict(N=0), -2), (dict(N=1 << 31), -2), (dict(d=0), -2), (dict(d=(1 << 20) + 1, ldx=1 << 21, ldr=1 << 21), -2), (dict(ldx=99), -2),
    (dict(ldr=99), -2), (dict(ldx=(1 << 40) + 1), -2), (dict(x=X + 1), -3), (dict(y=Y + 1), -3), (dict(w=W + 2), -3), (dict(st=ST + 4), -3),
    (dict(eps=-1.0), -4), (dict(eps=float("nan")), -4), (dict(eps=float("inf")), -4), (dict(eps=1e300), -4),
    (dict(y=X + 2), -2), (dict(s=R), -2), (dict(s=Y + 700), -2), (dict(st=Y), -2), (dict(y=W), -2), (dict(y=X, r=None, s=None), -2),
])
def test_norm_refuses(lib, kw, status):
    assert _fwd(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def _bwd(lib, **kw):
    a = dict(s=S, dt=1, N=4, d=100, lds=100, w=W, gdt=0, rms=0, st=ST, dy=DY, lddy=100, ds=DS, ldds=100, dx=DX, dw=DW, db=DB, ws=WS,
             nbytes=1 << 20)
    a.update(kw)
    return lib.hylo_norm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(s=None), -1), (dict(st=None), -1), (dict(dy=None), -1), (dict(ws=None), -1), (dict(dt=-1), -2), (dict(gdt=2), -2),
    (dict(N=-1), -2), (dict(d=0), -2), (dict(lds=99), -2), (dict(lddy=99), -2), (dict(ldds=99), -2), (dict(dx=DX + 1), -3),
    (dict(dw=DW + 2), -3), (dict(ws=WS + 8), -3), (dict(nbytes=64), -5), (dict(dx=DY), -2), (dict(dx=S), -2), (dict(dw=DB), -2),
    (dict(dx=DS), -2), (dict(ws=DX, nbytes=1 << 20), -2), (dict(dw=W), -2), (dict(dx=ST), -2),
])
def test_norm_backward_refuses(lib, kw, status):
    assert _bwd(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def test_workspace(lib):
    q = _lib.hylo_norm_backward_workspace_bytes
    assert q(0, 8) == 0 and q(8, 0) == 0 and q(1, (1 << 20) + 1) == 0
    assert q(1, 8) == 2 * 4 * 8
    for d in (1, 64, 2048, 8192, 8193, 1 << 20):  # bounded whatever N is
        assert 0 < q(1 << 30, d) <= 64 << 20 and q(1 << 30, d) % (8 * d) == 0


def test_python_checks():
    x, w = torch.zeros(3, 16), torch.ones(16)
    for bad in (lambda: layer_norm(x), lambda: rms_norm(x, w),  # not on a GPU
                lambda: layer_norm(x.double()), lambda: layer_norm(x[:, :0]), lambda: layer_norm(torch.zeros(())),
                lambda: layer_norm(x, w[:8]), lambda: layer_norm(x, w, w[:8]), lambda: layer_norm(x, w.bfloat16()),
                lambda: layer_norm(x.bfloat16(), w, w.bfloat16()), lambda: rms_norm(x.bfloat16(), w.half()),
                lambda: rms_norm(x, w, residual=x[:2]), lambda: rms_norm(x, w, residual=x.half()),
                lambda: layer_norm(x, w.view(1, 16))):
        with pytest.raises(ValueError):
            bad()
