"""GPU parity of layer_norm and rms_norm, forward and gradients, against the fp64 oracle.

Tolerances, element by element, with u = 2^-24 (half a step of fp32) and h = eps / 2 of the type that a result is rounded to:
a sum over a row adds at most `depth` = max(32, d / 128) + 16 values one after another, so it is off by depth u of the sum of
magnitudes. That gives the mean, the variance (and half as much the deviation) and thereby xh; the rest follows by the formulas.
A product or sum in fp32 adds u each. Column sums add rows one after another within a CTA, then slices: bounded
by all rows behind one another where they are few, and N / 64 + 64 of them otherwise.
"""
import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import _lib, build, layer_norm, rms_norm
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rounding(ref, dtype):
    """Half a step of the type at ref (fp16: also of its subnormal numbers)."""
    return half_step(dtype) * np.abs(ref) + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -140)


def make(N, d, dtype, gain, bias, residual, pad=0, seed=0, shift=0.5):
    gen = torch.Generator("cuda").manual_seed(seed)
    draw = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731

    def rows(x):
        buf = torch.full((N, d + pad), float("nan"), dtype=dtype, device="cuda")
        buf[:, :d] = x
        return buf[:, :d]

    x = rows(draw(N, d) * torch.exp(0.5 * draw(N, 1)) + shift)
    r = rows(0.5 * draw(N, d)) if residual else None
    gdt = None if gain is None else dtype if gain == "same" else torch.float32
    w = (1 + 0.2 * draw(d)).to(gdt) if gain else None
    b = (0.3 * draw(d)).to(gdt) if bias else None
    return x, r, w, b, rows(draw(N, d)), rows(draw(N, d)) if residual else None


def run(x, r, w, b, eps, rms):
    out = rms_norm(x, w, eps=eps, residual=r) if rms else layer_norm(x, w, b, eps=eps, residual=r)
    return out if r is not None else (out, None)


class Bounds:
    def __init__(self, s, w, b, eps, rms):
        self.s, self.w, self.rms = s, w, rms
        d = s.shape[1]
        self.depth = depth = max(32, d / 128) + 16
        self.y, mu, r = oo.norm(s, w, b, eps, rms)
        self.r = r
        dmu = 0.0 if rms else depth * U * np.abs(s).mean(1, keepdims=True) + U * np.abs(mu)
        self.xh = (s - mu) * r
        rel_r = (depth + 8) * U / 2 + 4 * U + (r * dmu) ** 2  # the variance's sum, its factor, the root
        self.dxh = r * dmu + np.abs(self.xh) * (rel_r + 3 * U)
        self.rel_r = rel_r
        ww = 1.0 if w is None else np.abs(w)
        self.dy = ww * self.dxh + 2 * U * np.abs(self.xh) * ww + U * np.abs(self.y)

    def grads(self, dy):
        """Bounds of (dx before dsum, dweight, dbias)."""
        N = dy.shape[0]
        g = dy if self.w is None else dy * self.w
        mean = lambda v: np.abs(v).mean(1, keepdims=True)  # noqa: E731
        c1, c2 = (g * self.xh).mean(1, keepdims=True), 0.0 if self.rms else g.mean(1, keepdims=True)
        dc1 = (self.depth + 4) * U * mean(g * self.xh) + (np.abs(g) * self.dxh).mean(1, keepdims=True)
        dc2 = 0.0 if self.rms else (self.depth + 4) * U * mean(g)
        inner = np.abs(g) + np.abs(c2) + np.abs(self.xh * c1)
        dx = self.r * (4 * U * inner + dc2 + np.abs(self.xh) * dc1 + self.dxh * np.abs(c1)) + self.r * inner * self.rel_r
        rows = min(N, N / 64 + 64) + 8
        dw = (np.abs(dy) * self.dxh).sum(0) + rows * U * np.abs(dy * self.xh).sum(0)
        return dx, dw, rows * U * np.abs(dy).sum(0)


def check(got, ref, bound, dtype, what):
    got = f64(got)
    assert got.shape == ref.shape, what
    tol = bound + rounding(np.abs(ref) + bound, dtype)
    worst = (np.abs(got - ref) / tol).max() if got.size else 0.0
    assert worst <= 1, (what, worst)


SIZES = [(1, 1), (5, 3), (7, 8), (2, 17), (3, 31), (4, 32), (9, 64), (33, 100), (6, 255), (5, 256), (3, 257), (333, 520),
         (4, 1000), (3, 1001), (700, 2048), (5, 4096), (2, 8192), (3, 8200), (2, 16384), (2, 16392), (1, 32768), (2, 33001), (2, 70000)]


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,gain,bias,residual,pad", [
    ("bf16", "same", False, True, 0), ("bf16", "fp32", True, False, 8), ("fp32", "same", True, True, 0), ("fp16", "fp32", True, True, 3),
    ("fp16", None, False, False, 0), ("fp32", None, True, False, 1), ("bf16", "fp32", False, True, 1),
])
@pytest.mark.parametrize("N,d", SIZES)
def test_forward_and_gradients(N, d, dtype, gain, bias, residual, pad, rms):
    dtype, bias = DT[dtype], bias and not rms
    if gain is None and bias:
        gain = "fp32"
    eps = 1e-4
    x, r, w, b, dy, ds = make(N, d, dtype, gain, bias, residual, pad, seed=N + d)
    leaves = [t for t in (x, r, w, b) if t is not None]
    for t in leaves:
        t.requires_grad_()
    y, total = run(x, r, w, b, eps, rms)
    assert y.is_contiguous() and y.dtype == dtype
    s = f64(x)
    if residual:
        assert torch.equal(total, (x.float() + r.float()).to(dtype))
        s = f64(total)
    bounds = Bounds(s, f64(w), f64(b), eps, rms)
    check(y, bounds.y, bounds.dy, dtype, "y")
    grads = torch.autograd.grad([y] if total is None else [y, total], leaves, [dy] if ds is None else [dy, ds])
    grads = dict(zip([n for n, t in zip("xrwb", (x, r, w, b)) if t is not None], grads))
    rdx, rdw, rdb = oo.norm_grad(s, f64(w), eps, rms, f64(dy))
    bdx, bdw, bdb = bounds.grads(f64(dy))
    if residual:
        rdx = rdx + f64(ds)
        bdx = bdx + U * np.abs(rdx)
        assert torch.equal(grads["x"], grads["r"])
    check(grads["x"], rdx, bdx, dtype, "dx")
    if w is not None:
        check(grads["w"], rdw, bdw, w.dtype, "dw")
    if b is not None:
        check(grads["b"], rdb, bdb, b.dtype, "db")
    with torch.no_grad():  # the same bits without gradients
        assert torch.equal(run(x, r, w, b, eps, rms)[0], y)


def test_one_gradient_at_a_time_is_the_same():
    for d in (520, 2048, 9000):
        x, _, w, b, dy, _ = make(50, d, torch.float32, "same", True, False)
        full = None
        for wants in ((1, 1, 1), (1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1)):
            leaves = [t.detach().clone().requires_grad_(bool(q)) for t, q in zip((x, w, b), wants)]
            y = layer_norm(*leaves)
            got = torch.autograd.grad(y, [t for t in leaves if t.requires_grad], dy)
            if full is None:
                full = got
            assert all(torch.equal(a, f) for a, f in zip(got, [f for f, q in zip(full, wants) if q]))


def test_only_the_sum_is_used_and_only_the_norm():
    x, r, w, _, dy, ds = make(9, 64, torch.bfloat16, "same", False, True)
    for t in (x, r, w):
        t.requires_grad_()
    y, total = rms_norm(x, w, residual=r)
    gx, gr, gw = torch.autograd.grad(total, (x, r, w), ds, retain_graph=True, allow_unused=True)
    assert torch.equal(gx, ds) and torch.equal(gr, ds) and torch.count_nonzero(gw) == 0
    (gx,) = torch.autograd.grad(y, x, dy, retain_graph=True)
    both = torch.autograd.grad((y, total), x, (dy, torch.zeros_like(ds)))[0]
    assert torch.equal(gx, both)


def test_shapes_and_strides():
    x, _, w, b, _, _ = make(24, 40, torch.float32, "same", True, False)
    ref = layer_norm(x, w, b)
    assert torch.equal(layer_norm(x.view(2, 3, 4, 40), w, b), ref.view(2, 3, 4, 40))
    assert torch.equal(layer_norm(x[0], w, b), ref[0])
    assert torch.equal(layer_norm(x.T.contiguous().T, w, b), ref)          # column-major
    assert torch.equal(layer_norm(x[::3], w, b), ref[::3])
    assert torch.equal(layer_norm(x[:1].expand(5, 40), w, b), ref[:1].expand(5, 40))
    assert layer_norm(x[:0], w, b).shape == (0, 40) and layer_norm(x.view(2, 12, 40)[:, :0], w, b).shape == (2, 0, 40)
    off = torch.empty(24 * 40 + 1, device="cuda")[1:].view(24, 40).copy_(x)  # not 16-byte aligned
    assert (layer_norm(off, w, b) - ref).abs().max() < 1e-5
    wide = torch.stack([w, w], 1)[:, 0]                                     # a gain with a stride
    assert torch.equal(layer_norm(x, wide, b), ref)
    y = x.detach().requires_grad_()
    layer_norm(y, w, b).sum().backward()                                    # an expanded upstream gradient
    rdx, _, _ = oo.norm_grad(f64(x), f64(w), 1e-5, False, np.ones((24, 40)))
    bdx, _, _ = Bounds(f64(x), f64(w), f64(b), 1e-5, False).grads(np.ones((24, 40)))
    check(y.grad, rdx, bdx, torch.float32, "dx")
    e = x[:0].detach().requires_grad_()
    we = w.detach().requires_grad_()
    out = layer_norm(e, we, b)
    ge, gw = torch.autograd.grad(out, (e, we), torch.empty_like(out))
    assert ge.shape == (0, 40) and torch.count_nonzero(gw) == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("d", [100, 2048, 40000])
def test_far_means_and_constant_rows(d, rms):
    """A mean far above the deviation costs the mean's own error only; a row without deviation gives the bias."""
    x, _, w, b, dy, _ = make(6, d, torch.float32, "same", True, False, shift=300.0)
    b = None if rms else b
    x[3] = 7.0
    x[4] = 0.0
    y, _ = run(x, None, w, b, 1e-5, rms)
    bounds = Bounds(f64(x), f64(w), f64(b), 1e-5, rms)
    check(y, bounds.y, bounds.dy, torch.float32, "y")
    x.requires_grad_()
    dx = torch.autograd.grad(run(x, None, w, b, 1e-5, rms)[0], x, dy)[0]
    rdx, _, _ = oo.norm_grad(f64(x), f64(w), 1e-5, rms, f64(dy))
    check(dx, rdx, bounds.grads(f64(dy))[0], torch.float32, "dx")


@pytest.mark.parametrize("d", [64, 300, 4096, 9000])
def test_rows_that_are_not_finite_stay_alone(d):
    x, _, w, _, dy, _ = make(40, d, torch.bfloat16, "same", False, False)
    ref = rms_norm(x, w)
    x[7, d // 2], x[21, 0] = float("nan"), float("inf")
    x.requires_grad_()
    y = rms_norm(x, w)
    (dx,) = torch.autograd.grad(y, x, dy)
    keep = [i for i in range(40) if i not in (7, 21)]
    assert torch.equal(y[keep], ref[keep]) and torch.isnan(y[7]).all() and torch.isnan(y[21, 0])
    assert torch.isfinite(dx[keep].float()).all()


def test_gradient_against_differences():
    x, r, w, b, dy, ds = make(3, 19, torch.float32, "same", True, True)
    for t in (x, r, w, b):
        t.requires_grad_()
    grads = torch.autograd.grad(layer_norm(x, w, b, residual=r), (x, r, w, b), (dy, ds))

    def f(parts):  # in 64 bits
        xx, rr, ww, bb = parts
        s = xx + rr
        return (oo.norm(s, ww, bb, 1e-5, False)[0] * f64(dy)).sum() + (s * f64(ds)).sum()

    parts = [f64(t) for t in (x, r, w, b)]
    for k, g in enumerate(grads):
        g = f64(g)
        for i in np.ndindex(parts[k].shape):
            e = [p.copy() for p in parts]
            e[k][i] += 1e-5
            up = f(e)
            e[k][i] -= 2e-5
            assert abs((up - f(e)) / 2e-5 - g[i]) < 1e-4 * (1 + abs(g[i]))


def test_rows_behind_the_last_and_far_rows():
    """Nothing behind [N, d] is written; rows whose offsets pass 32 bits."""
    N, d = 5, 72
    x, _, w, _, _, _ = make(N, d, torch.bfloat16, "same", False, False)
    y = torch.full((N + 2, d), 3.0, dtype=torch.bfloat16, device="cuda")
    st = torch.full((N + 2, 2), 3.0, device="cuda")
    _lib.hylo_norm(x, None, w, None, True, 1e-6, None, y[:N], st[:N])
    assert torch.equal(y[:N], rms_norm(x, w)) and (y[N:] == 3).all() and (st[N:] == 3).all()
    step = (1 << 31) + 8
    big = torch.empty(2 * step + d, dtype=torch.bfloat16, device="cuda").as_strided((3, d), (step, 1))
    big.copy_(x[:3])
    assert torch.equal(rms_norm(big, w), y[:3])
    big.requires_grad_()
    dy = torch.ones(3, d, dtype=torch.bfloat16, device="cuda")
    small = x[:3].detach().clone().requires_grad_()
    a = torch.autograd.grad(rms_norm(big, w), big, dy)[0]
    assert torch.equal(a, torch.autograd.grad(rms_norm(small, w), small, dy)[0])


def test_many_rows():
    """More rows than 2^31 / d and than any grid: every row as in a call of its own."""
    N, d = 300_001, 8192
    x = torch.randn(64, d, device="cuda").bfloat16().repeat(N // 64 + 1, 1)[:N]
    y = rms_norm(x)
    ref = rms_norm(x[:64])
    for lo in range(0, N, 64 * 1000):
        part = y[lo:lo + 64 * 1000]
        assert torch.equal(part, ref.repeat(1000, 1)[:part.shape[0]])


@pytest.mark.parametrize("N,d", [(5000, 256), (3000, 2048), (700, 8192), (300, 20000)])
def test_repeats_bit_for_bit_also_on_another_stream_and_in_a_graph(N, d):
    x, r, w, b, dy, ds = make(N, d, torch.bfloat16, "fp32", True, True)
    for t in (x, r, w, b):
        t.requires_grad_()

    def step():
        y, s = layer_norm(x, w, b, residual=r)
        return (y, s) + torch.autograd.grad((y, s), (x, r, w, b), (dy, ds))

    ref = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(ref, other))
    leaves = [t.detach().clone().requires_grad_() for t in (x, r, w, b)]  # leaves of their own: no eager graph of theirs lives

    def captured():
        y, s = layer_norm(leaves[0], leaves[2], leaves[3], residual=leaves[1])
        return (y, s) + torch.autograd.grad((y, s), leaves, (dy, ds))

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured()
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, c) for a, c in zip(ref, out))


def test_second_derivatives_and_tangents_are_refused():
    x, _, w, _, _, _ = make(4, 16, torch.float32, "same", False, False)
    x.requires_grad_()
    g = torch.autograd.grad(layer_norm(x, w).square().sum(), x, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="differentiable once"):
        g.sum().backward()
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            rms_norm(torch.autograd.forward_ad.make_dual(x.detach(), torch.ones_like(x)), w)


def test_the_same_tensor_twice_and_gradients_of_their_own():
    x, r, w, _, dy, ds = make(20, 72, torch.float32, "same", False, True)
    a, b = (t.detach().clone().requires_grad_() for t in (x, x))
    y, s = rms_norm(a, w, residual=b)
    torch.autograd.backward((y, s), (dy, ds))
    assert torch.equal(a.grad, b.grad) and a.grad.data_ptr() != b.grad.data_ptr()  # one may be scaled in place without the other
    c = x.detach().clone().requires_grad_()
    y2, s2 = rms_norm(c, w, residual=c)
    torch.autograd.backward((y2, s2), (dy, ds))
    assert torch.equal(y2, y) and torch.equal(c.grad, 2 * a.grad)
    v = w.detach().clone().requires_grad_()  # one gain for two norms, as tied layers have it
    one = torch.autograd.grad(rms_norm(x, v), v, dy)[0] + torch.autograd.grad(rms_norm(r, v), v, dy)[0]
    two = torch.autograd.grad((rms_norm(x, v), rms_norm(r, v)), v, (dy, dy))[0]
    assert torch.equal(one, two)
    with torch.inference_mode():
        assert torch.equal(rms_norm(x, w), rms_norm(x.clone(), w))


def test_two_threads_with_a_stream_each():
    import threading
    jobs = []
    for i, d in enumerate((520, 6000)):
        x, _, w, b, dy, _ = make(300, d, torch.bfloat16, "fp32", True, False, seed=i)
        x, w, b = (t.detach().clone().requires_grad_() for t in (x, w, b))
        y = layer_norm(x, w, b)
        jobs.append((x, w, b, dy, (y,) + torch.autograd.grad(y, (x, w, b), dy)))
    torch.cuda.synchronize()
    wrong = []

    def work(job):
        x, w, b, dy, ref = job
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                y = layer_norm(x, w, b)
                got = (y,) + torch.autograd.grad(y, (x, w, b), dy)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(p, q) for p, q in zip(got, ref)):
                    wrong.append(x.shape)

    threads = [threading.Thread(target=work, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
