"""GPU parity of orthogonalize and muon_step against the fp64 oracle.

Tolerances. An fp16 number is off by at most 2^-11 of itself and 1.0e-4 of it in the root mean square. With spectral norms
|X| <= 1.2, |b| = 4.8, |c| = 2, a step takes the roundings of X (three times: twice in A, once in B X), A and B into the next
X with a weight of |B| + 3 (|b| + 2 |c| |A|) |X|^2 + |B| <= 45 of its Frobenius norm, worst case: 45 x 1.0e-4 = 4.5e-3, so
5e-3 of the norm (a step's errors are not amplified by the next beyond that: where the slope of a x + b x^3 + c x^5 is above 1,
at small singular values, B is small and X is kept in two terms). After one step the oracle that rounds where the kernels round
differs from them only by fp32 sums, which flip a rounding in about (K / 16) 2^-24 / 2^-11 of the elements, 2 % at K = 2048:
sqrt(0.02) 4.5e-3 = 6e-4, so 1e-3. After more steps it says no more than the exact one: a difference of 1e-5 flips 2 % of the next
step's roundings, that step's difference of 6e-4 all of them, which leaves two independent sets of roundings.
"""
import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import Muon, _lib, build, grad_norm, muon_step, orthogonalize
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EXACT, SCHEME, U = 5e-3, 1e-3, 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def f64(t):
    return t.detach().double().cpu().numpy()


def matrix(rows, cols, seed=0, kind="gauss"):
    gen = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    if kind == "low":
        k = max(1, min(rows, cols) // 16)
        x = 0.05 * x + torch.randn(rows, k, generator=gen, device="cuda") @ torch.randn(k, cols, generator=gen, device="cuda")
    return x


def near(got, x, out, coefficients=(oo.MUON,) * 5, eps=1e-7):
    """`got` against the exact steps (one step: and against the scheme's), in the Frobenius norm, with one rounding to the
    result's type."""
    h = torch.finfo(out).eps / 2
    got = f64(got)
    refs = [(oo.orthogonalize(x, coefficients, eps), EXACT)]
    if len(coefficients) == 1:
        refs.append((oo.orthogonalize_fp16(x, coefficients, eps), SCHEME))
    for ref, tol in refs:
        err, norm = np.linalg.norm(got - ref), np.linalg.norm(ref)
        assert err <= (tol + h) * norm + 2.0 ** -25 * np.sqrt(ref.size), (err / norm, tol)


SIZES = [(1, 1), (1, 7), (9, 1), (2, 3), (63, 65), (64, 64), (65, 63), (255, 256), (257, 256), (256, 257), (520, 128), (300, 1000),
         (1000, 300), (513, 700), (128, 4096), (1, 100_000), (70_000, 2), (100, 8200), (300, 17_000), (1030, 1029), (2048, 512)]


@pytest.mark.parametrize("kind", ["gauss", "low"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols, kind):
    x = matrix(rows, cols, rows + cols, kind)
    y = orthogonalize(x, dtype=torch.float16)
    _lib.hylo_kl_sync_status()
    assert y.shape == x.shape and y.is_contiguous() and y.dtype == torch.float16
    near(y, f64(x), torch.float16)
    near(orthogonalize(x, steps=1, dtype=torch.float16), f64(x), torch.float16, (oo.MUON,))


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("out", ["bf16", "fp16"])
def test_types_strides_and_lists(dtype, out):
    """A list of matrices whose sums are not split gives what each gives alone, bit for bit, whatever its strides."""
    dt, out = DT[dtype], DT[out]
    mats = []
    for i, (r, c, pad) in enumerate([(70, 300, 0), (300, 70, 3), (257, 300, 1), (64, 64, 8), (1, 50, 5), (50, 1, 5), (400, 512, 0)]):
        buf = torch.full((r, c + pad), float("nan"), device="cuda", dtype=dt)
        buf[:, :c] = matrix(r, c, i).to(dt)
        mats.append(buf[:, :c])
    ys = orthogonalize(mats, dtype=out)
    for x, y in zip(mats, ys):
        assert y.dtype == out and y.is_contiguous()
        near(y, f64(x), out)
        assert torch.equal(orthogonalize(x.contiguous(), dtype=out), y)
    y = orthogonalize(mats[0].T, dtype=out)  # read by its columns
    assert y.is_contiguous() and torch.equal(y, ys[0].T)
    every = mats[6][::2, ::2]                # neither rows nor columns have unit stride
    assert torch.equal(orthogonalize(every, dtype=out), orthogonalize(every.contiguous(), dtype=out))
    stack = torch.stack([matrix(40, 90, i).to(dt) for i in range(6)])
    one = orthogonalize(stack, dtype=out)
    two = orthogonalize(stack.view(2, 3, 40, 90), dtype=out)
    turned = orthogonalize(stack.transpose(1, 2), dtype=out)
    for i in range(6):
        ref = orthogonalize(stack[i], dtype=out)
        assert torch.equal(one[i], ref) and torch.equal(two[i // 3, i % 3], ref) and torch.equal(turned[i], ref.T)
    assert orthogonalize(stack[:0], dtype=out).shape == (0, 40, 90) and orthogonalize([], dtype=out) == []
    assert orthogonalize(torch.empty(0, 5, device="cuda"), dtype=out).shape == (0, 5)


def test_many_matrices_in_several_groups():
    mats = [matrix(10 + i % 7, 20 + i % 11, i) for i in range(150)]
    ys = orthogonalize(mats, dtype=torch.float16)
    for x, y in zip(mats[::13], ys[::13]):
        near(y, f64(x), torch.float16)
    big = [matrix(1024, 8192, i) for i in range(24)]  # 24 x 52 MiB of workspace: more than one group's
    ys = orthogonalize(big, dtype=torch.float16)
    again = orthogonalize(big, dtype=torch.float16)
    assert all(torch.equal(a, b) for a, b in zip(ys, again))
    near(ys[23], f64(big[23]), torch.float16)


@pytest.mark.parametrize("shapes", [[(100, 9000)], [(300, 8129), (1030, 8250)], [(5, 70_000), (600, 8191), (40, 50)], [(9000, 1100)],
                                    [(1, 300_000)], [(20, 600_000)]])
def test_split_sums(shapes):
    """Sums of A in parts, some of them longer than the tensor cores take at a time; bit for bit the same every time."""
    xs = [matrix(r, c, r) for r, c in shapes]
    ys = orthogonalize(xs, dtype=torch.float16)
    _lib.hylo_kl_sync_status()
    for x, y in zip(xs, ys):
        near(y, f64(x), torch.float16)
    near(orthogonalize(xs, steps=1, dtype=torch.float16)[0], f64(xs[0]), torch.float16, (oo.MUON,))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(ys, orthogonalize(xs, dtype=torch.float16)))


@pytest.mark.parametrize("k,steps", [((1.5, -0.5, 0.0), 12), ((2.0, -1.5, 0.5), 6), ((3.4445, -4.775, 2.0315), 1)])
def test_other_coefficients(k, steps):
    x = matrix(90, 200, 5)
    y = orthogonalize(x, steps=steps, coefficients=k, dtype=torch.float16)
    near(y, f64(x), torch.float16, (k,) * steps)
    each = [(4.0, -6.0, 2.5), (3.0, -3.0, 1.0), (2.0, -1.5, 0.5)]
    y = orthogonalize(x, steps=3, coefficients=each, eps=1.0, dtype=torch.float16)
    near(y, f64(x), torch.float16, each, 1.0)


@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e12, 1e30, 2.0 ** 127])
def test_any_magnitude(size):
    """Squares that leave fp32's range; eps = 0 so that small ones are scaled up too."""
    for r, c in ((40, 70), (300, 200)):
        x = matrix(r, c, 1)
        x = x / x.abs().max() * size
        near(orthogonalize(x, eps=0.0, dtype=torch.float16), f64(x) / size, torch.float16, eps=0.0)


def test_zeros_and_what_is_not_finite():
    zeros, good = torch.zeros(300, 90, device="cuda"), matrix(130, 70, 2)
    bad = [matrix(300, 280, 3), matrix(300, 280, 3), matrix(2, 5, 4)]
    bad[0][299, 279], bad[1][0, 0], bad[2][0, 1] = float("nan"), float("inf"), -float("inf")
    ys = orthogonalize([bad[0], good, zeros, bad[1], good, bad[2]])
    assert torch.equal(ys[1], orthogonalize(good)) and torch.equal(ys[4], ys[1]) and torch.count_nonzero(ys[2]) == 0
    assert all(torch.isnan(ys[i]).all() for i in (0, 3, 5))
    assert torch.count_nonzero(orthogonalize(zeros, eps=0.0)) == 0


def test_orthogonal_and_diagonal_matrices():
    q = torch.linalg.qr(torch.randn(300, 300, dtype=torch.float64, device="cuda"))[0].float()
    near(orthogonalize(q, dtype=torch.float16), f64(q), torch.float16)
    d = torch.diag(torch.logspace(0, -6, 200, device="cuda"))
    y = orthogonalize(d, dtype=torch.float16)
    near(y, f64(d), torch.float16)
    assert torch.count_nonzero(y - torch.diag(torch.diag(y))) == 0


def test_repeats_also_on_another_stream_in_a_graph_and_in_two_that_share_a_pool():
    mats = [matrix(300, 500, 1), matrix(1000, 70, 2), matrix(600, 600, 3)]
    ref = orthogonalize(mats)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = orthogonalize(mats)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(ref, other))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    with torch.cuda.graph(graphs[0]):
        outs.append(orthogonalize(mats))
    with torch.cuda.graph(graphs[1], pool=graphs[0].pool()):
        outs.append(orthogonalize(mats[::-1]))
    for _ in range(2):
        graphs[0].replay()
        a = [t.clone() for t in outs[0]]
        graphs[1].replay()
        b = [t.clone() for t in outs[1]][::-1]
        assert all(torch.equal(x, y) and torch.equal(x, z) for x, y, z in zip(ref, a, b))


def test_two_streams_at_once():
    xs = [matrix(700, 900, i) for i in range(2)]
    refs = [orthogonalize(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    ys = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                ys[i].append(orthogonalize(xs[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, r) for r, got in zip(refs, ys) for y in got)


def test_nothing_behind_a_result_is_written():
    x = matrix(37, 41, 6)
    buf = torch.full((37 * 41 + 64,), 5.0, dtype=torch.float16, device="cuda")
    import struct
    table = struct.pack("=" + _lib.ORTH_MATRIX, x.data_ptr(), buf.data_ptr(), 37, 41, 41)
    n = _lib.hylo_orthogonalize_workspace_bytes(table, 1)
    ws = torch.full((n + 256,), 77, dtype=torch.uint8, device="cuda")
    _lib.hylo_orthogonalize(table, 1, torch.float32, torch.float16, list(oo.MUON) * 5, 1e-7, ws[:n])
    assert torch.equal(buf[:37 * 41].view(37, 41), orthogonalize(x, dtype=torch.float16))
    assert (buf[37 * 41:] == 5).all() and (ws[n:] == 77).all()


# ------------------------------------------------------------------------------------------------- steps
def state(shapes, param, grad, seed=0):
    p, master, g, m = [], [], [], []
    for i, s in enumerate(shapes):
        gen = torch.Generator("cuda").manual_seed(seed + i)
        w = 0.02 * torch.randn(*s, generator=gen, device="cuda")
        p.append(w.clone() if param == "fp32" else w.bfloat16())
        master.append(w if param == "master" else p[-1].float())
        g.append((1e-3 * torch.randn(*s, generator=gen, device="cuda")).to(DT[grad]))
        m.append(4e-4 * torch.randn(*s, generator=gen, device="cuda"))
    return p, (master if param == "master" else None), g, m


def rounded_up(w32, bits16):
    return ((w32.view(np.uint32) + bits16.astype(np.uint32)) & np.uint32(0xFFFF0000)).view(np.float32)


@pytest.mark.parametrize("param", ["fp32", "master", "bf16"])
@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("nesterov,adjust", [(True, "rms"), (False, "shape")])
def test_step(param, grad, nesterov, adjust):
    """Momentum to fp32 roundings, parameters to the orthogonalised update's accuracy, bf16 alone to the step between
    two bf16 numbers besides (2^-7 at most, a half in the root mean square)."""
    shapes = [(70, 300), (300, 70), (3, 40, 64), (1, 33), (257, 255)]
    p, master, g, m = state(shapes, param, grad)
    before = [f64(t) for t in (master or p)], [f64(t) for t in g], [f64(t) for t in m]
    lr, wd = [0.02, 0.01, 0.02, 0.03, 0.02], 0.1
    muon_step(p, g, m, lr=lr, momentum=0.9, nesterov=nesterov, weight_decay=wd, adjust=adjust, masters=master, seed=3)
    _lib.hylo_kl_sync_status()
    for i, s in enumerate(shapes):
        rows, cols = s[-2:]
        scale = np.sqrt(max(1, rows / cols)) if adjust == "shape" else 0.2 * np.sqrt(max(rows, cols))
        w, gg, mm = (f64(x).reshape(-1, rows, cols) if isinstance(x, torch.Tensor) else x.reshape(-1, rows, cols)
                     for x in (before[0][i], before[1][i], before[2][i]))
        for b in range(w.shape[0]):
            rw, rm = oo.muon(w[b], gg[b], mm[b], lr=lr[i], momentum=0.9, nesterov=nesterov, weight_decay=wd, scale=scale)
            got_m = f64(m[i]).reshape(-1, rows, cols)[b]
            assert np.all(np.abs(got_m - rm) <= 4 * U * (np.abs(mm[b]) + np.abs(gg[b])))
            o = (w[b] * (1 - lr[i] * wd) - rw)
            tol = (EXACT + 2.0 ** -11) * np.linalg.norm(o) + 4 * U * np.linalg.norm(w[b])
            got = f64((master or p)[i]).reshape(-1, rows, cols)[b]
            assert np.linalg.norm(got - rw) <= tol + (2.0 ** -7 * np.linalg.norm(rw) if param == "bf16" else 0)
            if param == "master":
                assert torch.equal(p[i], master[i].bfloat16())


@pytest.mark.parametrize("shape", [(70, 300), (301, 67), (512, 512), (2, 30, 40)])
@pytest.mark.parametrize("param", ["fp32", "bf16"])
def test_step_without_momentum_to_the_last_bit(shape, param):
    """momentum = 0: the update is the gradient, so O is orthogonalize's; every element of the step then has a few fp32
    roundings, and a bf16 parameter is one of the roundings of a number within them."""
    p, _, g, m = state([(5, 7), shape], param, "fp32")
    w = [t.float().clone() for t in p]
    os = [orthogonalize(t, dtype=torch.float16).float() for t in g]
    muon_step(p, g, m, lr=0.5, momentum=0.0, weight_decay=0.1, adjust=None, seed=11)
    pos = 0
    for i in range(2):
        assert torch.equal(m[i], g[i])
        ref = f64(w[i]) * np.float64(np.float32(1 - 0.05)) - 0.5 * f64(os[i])
        # the returned O is rounded to fp16's subnormal numbers, half a step of which is 2^-25; the step's O is scaled
        tol = 2 * U * (np.abs(ref) + np.abs(0.5 * f64(os[i]))) + 0.5 * 2.0 ** -25
        if param == "fp32":
            assert np.all(np.abs(f64(p[i]) - ref) <= tol)
        else:
            got, n = p[i].float().cpu().numpy(), ref.shape[-2] * ref.shape[-1]
            for k in range(ref.size // n):  # rounding with given random bits is monotone; every matrix starts at a multiple of 256
                bits = oo.random_bits(11, pos, n).reshape(ref.shape[-2:])
                bits = ((bits * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)) >> np.uint64(16)
                at = (lambda t: t.reshape(-1, *ref.shape[-2:])[k])  # noqa: E731
                lo, hi = (rounded_up((at(ref) + s * at(tol)).astype(np.float32), bits) for s in (-1, 1))
                assert np.all((lo <= at(got)) & (at(got) <= hi))
                pos += -(-n // 256) * 256
            continue
        pos += -(-ref.size // 256) * 256


def test_norm_clips_and_skips():
    p, _, g, m = state([(64, 90), (90, 64)], "fp32", "fp32")
    norm = grad_norm(g)
    q, n = [t.clone() for t in p], [t.clone() for t in m]
    muon_step(p, g, m, lr=0.1, norm=norm, max_norm=0.01, grad_scale=0.5)
    c = min(1.0, 0.01 / (0.5 * norm.item() + 1e-6)) * 0.5
    for a, b, x in zip(m, n, g):
        assert np.all(np.abs(f64(a) - (0.95 * f64(b) + 0.05 * c * f64(x))) <= 8 * U * (np.abs(f64(b)) + np.abs(c * f64(x))))
    before = [t.clone() for t in p + m]
    for bad in (float("nan"), float("inf")):
        muon_step(p, g, m, lr=0.1, norm=torch.tensor([bad], device="cuda"))
        assert all(torch.equal(a, b) for a, b in zip(before, p + m))
    assert not torch.equal(q[0], p[0])


def test_optimiser_class_groups_states_and_versions():
    torch.manual_seed(0)
    a, b = (torch.randn(60, 80, device="cuda").bfloat16().requires_grad_() for _ in range(2))
    opt = Muon([{"params": [a]}, {"params": [b], "lr": 0.05}], lr=0.01, weight_decay=0.1, max_norm=1.0)
    loss = (a.float() @ b.float().T).square().mean()
    loss.backward()
    w = [t.clone() for t in opt.masters]
    opt.step()
    assert opt.steps == 1 and opt.last_norm.item() > 0
    c = min(1.0, 1.0 / (opt.last_norm.item() + 1e-6))
    for t, w0, lr, x in zip(opt.masters, w, (0.01, 0.05), (a, b)):
        rw, _ = oo.muon(f64(w0), c * f64(x.grad), np.zeros((60, 80)), lr=lr, momentum=0.95, nesterov=True, weight_decay=0.1, scale=1.0)
        assert np.linalg.norm(f64(t) - rw) <= 6e-3 * np.linalg.norm(f64(w0) * (1 - lr * 0.1) - rw) + 4 * U * np.linalg.norm(rw)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y = (a * a).sum()
        opt.step()
        y.backward()
    saved = {k: [t.clone() for t in v] if isinstance(v, list) else v for k, v in opt.state_dict().items()}
    opt.step()
    opt.load_state_dict(saved)
    assert opt.steps == 2 and torch.equal(opt.momenta[0], saved["momenta"][0])
    with pytest.raises(ValueError):
        opt.load_state_dict({**saved, "masters": None})


def test_a_captured_step_is_refused():
    p, _, g, m = state([(64, 64)], "fp32", "fp32")
    muon_step(p, g, m, lr=0.1)
    before = p[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        try:
            with pytest.raises(_lib.HyloError, match="HYLO_ERR_CAPTURE"):
                muon_step(p, g, m, lr=0.1)
        finally:
            graph.capture_end()
    torch.cuda.synchronize()
    assert torch.equal(before, p[0])


def test_overlapping_arrays_are_refused():
    w = torch.zeros(64, 64, device="cuda")
    g, m = torch.ones(64, 64, device="cuda"), torch.zeros(64, 64, device="cuda")
    for args in (([w, w], [g, g], [m, m.clone()]), ([w], [w], [m]), ([w], [g], [w]), ([w], [m], [m])):
        with pytest.raises(_lib.HyloError, match="overlap"):
            muon_step(*args, lr=0.1)


def test_vectors_as_matrices_and_a_batch_of_experts():
    """Parameters of one row, of one column, and a batch, with and without masters, in one optimiser."""
    torch.manual_seed(1)
    shapes = [(1, 300), (300, 1), (4, 24, 50), (2, 2, 16, 16), (0, 8)]
    for masters in (True, False):
        ps = [torch.randn(s, device="cuda").bfloat16().requires_grad_() for s in shapes]
        opt = Muon(ps, lr=0.1, masters=masters, momentum=0.0, nesterov=False, adjust=None)
        gs = [torch.randn_like(p) for p in ps]
        before = [p.detach().clone() for p in ps]
        opt.step(gs)
        for p, b, g in zip(ps, before, gs):
            want = f64(b) - 0.1 * f64(orthogonalize(g, dtype=torch.float16))
            # half a bf16 step to nearest, a whole one (2^-7) rounded at random; fp32 roundings besides
            unit = 2.0 ** -8 if masters else 2.0 ** -7
            assert np.all(np.abs(f64(p) - want) <= unit * np.abs(want) * (1 + 2.0 ** -7) + 1e-6)
