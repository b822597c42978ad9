"""Scratch of head_logprobs: the forward asks for what the forward needs, the backward for the gradients that are wanted."""
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, head_logprobs


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return _lib.load()


def test_sizes():
    fwd, bwd, both = (_lib.hylo_head_logprobs_forward_workspace_bytes, _lib.hylo_head_logprobs_backward_workspace_bytes,
                      _lib.hylo_head_logprobs_workspace_bytes)
    assert fwd(8192, 4096, 128256) == 8192 * (4 + 2 * 32 * 16)  # logits of the tokens, two sums per segment
    assert fwd(1 << 20, 2048, 128256) == both(1 << 20, 2048, 128256)
    bf, ring = dict(grad_dtype=torch.bfloat16), 3 * 4096 * 5376 * 2
    assert bwd(8192, 2048, 128256, **bf) == both(8192, 2048, 128256, **bf) == ring + 256 + (8192 + 128256) * 2048 * 4
    assert bwd(8192, 2048, 128256, want_dW=False, **bf) == ring + 256 + 8192 * 2048 * 4
    assert bwd(8192, 2048, 128256, want_dh=False, **bf) == ring + 256 + 128256 * 2048 * 4
    assert bwd(4096, 2048, 128256, want_dh=False, **bf) == ring + 256
    assert bwd(1024, 2048, 128256, want_dh=False) == 3 * 1024 * 12288 * 2 + 256
    assert bwd(8192, 2048, 128256) == ring + 256  # fp32 gradients are their own sums
    for sizes in ((0, 64, 10), (1, 60, 10), (1, 64, 0)):
        assert fwd(*sizes) == 0 and bwd(*sizes) == 0
    assert bwd(16, 64, 10, want_dh=False, want_dW=False) == 0 and bwd(16, 64, 10, grad_dtype=torch.float16) == 0
    for n in (1, 7, 300, 1024, 1025, 5000):
        for split in (False, True):
            for dt in (torch.float32, torch.bfloat16):
                a = [bwd(n, 512, 32000, 0, split, dt, *w) for w in ((True, True), (True, False), (False, True))]
                assert a[0] >= max(a[1:]) and max(a[0], fwd(n, 512, 32000)) == both(n, 512, 32000, 0, split, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("N,d,V", [(1, 4096, 32000), (8192, 512, 32000)])
def test_scoring_takes_no_more_than_the_forward_needs(N, d, V):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W, h = (torch.randn(n, d, device="cuda").bfloat16() for n in (V, N))
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    for x in (h, h.clone().requires_grad_()):
        head_logprobs(x, W, t)
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        start = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        r = head_logprobs(x, W, t)
        peak = torch.cuda.max_memory_allocated() - start
        # the results and the allocator's rounding of each tensor besides
        assert peak <= _lib.hylo_head_logprobs_forward_workspace_bytes(N, d, V) + 3 * (4 * N + 512) + 512, peak
        del r


@pytest.mark.gpu
@pytest.mark.parametrize("N,d,V", [(8, 4096, 32000), (100, 64, 5003), (1500, 520, 5003), (5000, 64, 1000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("want", [(True, False), (False, True)])
def test_a_workspace_of_exactly_the_size_is_enough(N, d, V, dtype, split, want):
    """One gradient in a workspace of its own size is bit for bit that of both, and nothing behind the workspace is written."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    gen = torch.Generator("cuda").manual_seed(N)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    h, W = rnd(N, d).bfloat16(), (rnd(V, d) * 0.05).bfloat16()
    t, gl, ge = torch.randint(0, V, (N,), generator=gen, device="cuda"), rnd(N), rnd(N)
    logp, ent, lse = (torch.empty(N, device="cuda") for _ in range(3))
    n = _lib.hylo_head_logprobs_forward_workspace_bytes(N, d, V)
    ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    _lib.hylo_head_logprobs(h, W, t, 1.0, logp, ent, lse, ws[:n])
    assert torch.all(ws[n:] == 0x5A)
    out = []
    for w in ((True, True), want):
        n = _lib.hylo_head_logprobs_backward_workspace_bytes(N, d, V, 4096, split, dtype, *w)
        ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        dh, dW = (torch.empty(s, d, dtype=dtype, device="cuda") if x else None for s, x in zip((N, V), w))
        _lib.hylo_head_logprobs_backward(h, W, t, 1.0, 4096, lse, ent, gl, ge, dh, dW, ws[:n], split_g=split)
        assert torch.all(ws[n:] == 0x5A)
        out.append((dh, dW))
        with pytest.raises(_lib.HyloError):
            _lib.hylo_head_logprobs_backward(h, W, t, 1.0, 4096, lse, ent, gl, ge, dh, dW, ws[:n - 256], split_g=split)
    for a, b in zip(*out):
        assert b is None or torch.equal(a, b)
    _lib.hylo_kl_sync_status()
