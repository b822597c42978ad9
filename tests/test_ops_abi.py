"""Refusals of the operators in include/hylo_ops.h: the C entry points with bad arguments (these calls never
reach the GPU) and the checks of the Python functions."""
import ctypes
import struct

import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build

FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def _fwd(lib, **kw):
    a = dict(z=FAKE, dt=1, N=4, V=100, ld=100, tau=1.0, tok=FAKE, k=5, logp=FAKE, ent=FAKE, lse=None, stats=FAKE,
             top=FAKE, ids=FAKE)
    a.update(kw)
    return lib.hylo_token_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), -1), (dict(tok=None), -1), (dict(logp=None), -1), (dict(top=None), -1), (dict(ids=None), -1),
    (dict(dt=3), -2), (dict(dt=-1), -2), (dict(N=0), -2), (dict(V=0), -2), (dict(V=1 << 31, ld=1 << 31), -2),
    (dict(ld=99), -2), (dict(k=-1), -2), (dict(k=65), -2), (dict(V=4, k=5), -2), (dict(z=FAKE + 1), -3),
    (dict(dt=0, z=FAKE + 2), -3), (dict(tok=FAKE + 4), -3), (dict(stats=FAKE + 4), -3), (dict(ids=FAKE + 4), -3),
    (dict(tau=0.0), -4), (dict(tau=-1.0), -4), (dict(tau=float("nan")), -4), (dict(tau=float("inf")), -4),
    (dict(tau=1e-45), -4),
])
def test_token_logprobs_refuses(lib, kw, status):
    assert _fwd(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def _bwd(lib, **kw):
    a = dict(z=FAKE, dt=1, N=4, V=100, ld=100, tau=1.0, tok=FAKE, stats=FAKE, ent=FAKE, gl=FAKE, ge=FAKE, dz=FAKE, ldd=100)
    a.update(kw)
    return lib.hylo_token_logprobs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(z=None), -1), (dict(stats=None), -1), (dict(dz=None), -1), (dict(ent=None), -1), (dict(ldd=99), -2),
    (dict(N=-1), -2), (dict(dz=FAKE + 1), -3), (dict(stats=FAKE + 4), -3), (dict(gl=FAKE + 2), -3), (dict(tau=0.0), -4),
])
def test_token_logprobs_backward_refuses(lib, kw, status):
    assert _bwd(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def _norm(lib, grads=(FAKE,), sizes=(8,), count=None, dt=0, norm=FAKE, ws=FAKE, nbytes=1 << 20):
    n = len(grads)
    return lib.hylo_grad_norm((ctypes.c_uint64 * max(n, 1))(*grads), (ctypes.c_int64 * max(n, 1))(*sizes),
                              n if count is None else count, dt, norm, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(norm=None), -1), (dict(ws=None), -1), (dict(grads=(0,)), -1), (dict(count=-1), -2), (dict(sizes=(-1,)), -2),
    (dict(dt=2), -2), (dict(grads=(FAKE + 2,)), -3), (dict(ws=FAKE + 8), -3), (dict(nbytes=16), -5),
])
def test_grad_norm_refuses(lib, kw, status):
    assert _norm(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def _step(lib, tensors=None, pdt=0, gdt=0, bits=32, b1=0.9, b2=0.999, eps=1e-8, step=1, scale=1.0, norm=None,
          max_norm=1.0, **kw):
    t = dict(p=FAKE, g=FAKE, w=0, m=FAKE, v=FAKE, me=FAKE if bits == 8 else 0, ve=FAKE if bits == 8 else 0, n=10,
             lr=1e-3, wd=0.1)
    t.update(kw)
    rows = [t] if tensors is None else [{**t, **x} for x in tensors]
    table = b"".join(struct.pack("=" + _lib.ADAMW_TENSOR, *r.values()) for r in rows)
    return lib.hylo_adamw_step(table, len(rows), pdt, gdt, bits, b1, b2, eps, step, scale, norm, max_norm, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(p=0), -1), (dict(g=0), -1), (dict(m=0), -1), (dict(v=0), -1), (dict(bits=8, me=0), -1),
    (dict(bits=8, ve=0), -1), (dict(pdt=2), -2), (dict(gdt=2), -2), (dict(bits=16), -2), (dict(n=-1), -2),
    (dict(bits=8, eps=0.0), -2), (dict(b1=1.0), -2), (dict(b2=-0.1), -2), (dict(eps=-1.0), -2), (dict(step=0), -2), (dict(w=FAKE), -2),
    (dict(pdt=1, tensors=[dict(w=FAKE), dict(w=0)]), -2), (dict(b1=float("nan")), -2),
    (dict(p=FAKE + 2), -3), (dict(m=FAKE + 1), -3), (dict(lr=float("inf")), -4), (dict(wd=float("nan")), -4),
    (dict(scale=float("inf")), -4), (dict(norm=FAKE, max_norm=0.0), -4),
])
def test_adamw_refuses(lib, kw, status):
    assert _step(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def test_table_layout_is_the_headers():
    assert struct.calcsize("=" + _lib.ADAMW_TENSOR) == 80


def test_python_checks():
    from hybrid_upcycling_gb300 import AdamW, State8, adamw_step, grad_norm, token_logprobs
    z, t = torch.zeros(3, 10), torch.zeros(3, dtype=torch.int64)
    for bad in (lambda: token_logprobs(z, t),                       # not on a GPU
                lambda: token_logprobs(z.double(), t),
                lambda: token_logprobs(z, t[:2]),
                lambda: token_logprobs(z, t.int()),
                lambda: token_logprobs(z, t, top_k=11),
                lambda: token_logprobs(z[:, :0], t),
                lambda: grad_norm([]),
                lambda: grad_norm([z]),
                lambda: adamw_step([z], [z], [z], [z], step=1, lr=1e-3),
                lambda: adamw_step([z], [z], [z], [], step=1, lr=1e-3),
                lambda: AdamW([z], state_bits=4),
                lambda: AdamW([]),
                lambda: AdamW([z, z.bfloat16()])):
        with pytest.raises(ValueError):
            bad()
    s = State8.zeros_like(torch.zeros(257))
    assert s.codes.numel() == 257 and s.exponents.numel() == 2 and torch.all(s.values() == 0)


def _head(lib, **kw):
    a = dict(h=FAKE, W=FAKE, N=16, d=64, V=100, tau=1.0, tok=FAKE, logp=FAKE, ent=None, lse=None, ws=FAKE, nbytes=1 << 30)
    a.update(kw)
    return lib.hylo_head_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(h=None), -1), (dict(tok=None), -1), (dict(logp=None), -1), (dict(ws=None), -1), (dict(N=0), -2), (dict(d=60), -2),
    (dict(d=65544), -2), (dict(V=1 << 31), -2), (dict(h=FAKE + 8), -3), (dict(tok=FAKE + 4), -3), (dict(ws=FAKE + 16), -3),
    (dict(ent=FAKE + 2), -3), (dict(tau=0.0), -4), (dict(nbytes=64), -5),
])
def test_head_logprobs_refuses(lib, kw, status):
    assert _head(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def _head_bwd(lib, **kw):
    a = dict(h=FAKE, W=FAKE, N=16, d=64, V=100, tau=1.0, chunk=0, tok=FAKE, lse=FAKE, ent=FAKE, gl=FAKE, ge=FAKE, split=0, dt=0,
             dh=FAKE, dW=FAKE, ws=FAKE, nbytes=1 << 30)
    a.update(kw)
    return lib.hylo_head_logprobs_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(W=None), -1), (dict(lse=None), -1), (dict(dh=None, dW=None), -1), (dict(ent=None), -1), (dict(dh=None, ws=None), -1),
    (dict(N=-1), -2), (dict(d=12), -2), (dict(N=1 << 30, V=1 << 30), -2), (dict(dh=FAKE + 8), -3), (dict(gl=FAKE + 1), -3),
    (dict(tau=float("nan")), -4), (dict(nbytes=256), -5), (dict(dt=2), -2), (dict(dt=-1), -2), (dict(dt=1, dW=FAKE + 2), -3),
])
def test_head_logprobs_backward_refuses(lib, kw, status):
    if kw.get("N") == 1 << 30:
        kw = dict(kw, nbytes=1 << 62)
    assert _head_bwd(lib, **kw) == status
    assert lib.hylo_kl_last_error()


def test_head_workspace(lib):
    q = _lib.hylo_head_logprobs_workspace_bytes
    ring = 3 * 4096 * 5376 * 2
    assert q(4096, 2048, 128256) == ring + 256 and q(4096, 2048, 128256, split_g=True) == 2 * ring + 256
    assert q(1 << 20, 2048, 128256) == (1 << 20) * (4 + 2 * 32 * 16)
    assert q(1, 64, 256) == 3 * 256 * 256 * 2 + 256 + 256  # one part of dh
    assert q(1024, 2048, 128256) == 3 * 1024 * 12288 * 2 + 256 + 11 * 1024 * 2048 * 4  # 11 parts of 8 MiB
    assert q(512, 2048, 128256) == 3 * 512 * 24576 * 2 + 256 + 11 * 512 * 2048 * 4  # two of a block
    assert q(1025, 2048, 128256) == 3 * 1280 * 17408 * 2 + 256
    bf = dict(grad_dtype=torch.bfloat16)  # the fp32 sums: of dh, and of dW where the tokens are more than one block
    assert q(4096, 2048, 128256, **bf) == ring + 256 + 4096 * 2048 * 4
    assert q(4097, 2048, 128256, **bf) == ring + 256 + (4097 + 128256) * 2048 * 4
    assert q(4096, 2048, 128256, grad_dtype=torch.float16) == 0
    assert q(0, 64, 10) == 0 and q(1, 60, 10) == 0 and q(1, 64, 0) == 0


def test_head_python_checks():
    from hybrid_upcycling_gb300 import head_logprobs
    h, W, t = torch.zeros(3, 16).bfloat16(), torch.zeros(10, 16).bfloat16(), torch.zeros(3, dtype=torch.int64)
    for bad in (lambda: head_logprobs(h, W, t), lambda: head_logprobs(h.float(), W, t), lambda: head_logprobs(h, W[:, :8], t),
                lambda: head_logprobs(h, W, t[:2]), lambda: head_logprobs(h, W, t.int()),
                lambda: head_logprobs(h[:, :12], W[:, :12], t)):
        with pytest.raises(ValueError):
            bad()
