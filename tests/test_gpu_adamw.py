"""GPU parity of grad_norm and adamw_step against the fp64 oracle.

Tolerances, with u = 2^-24: an fp32 moment is two or three rounded operations: 4u of the sum of its terms'
magnitudes. The update m / (sqrt(v) rbc2 + eps) takes approximate square root and division (each within
2 ulp = 4u) and six rounded operations: 32u of itself; the parameter adds 2u of its own size. A code is
exactly the oracle's unless |x| 2^-e / step + random lies within 1e-4 steps of a whole number (the
fp32 moments are within 1e-6 of the oracle's, steps are at least 2^-4 of the value, and the square root doubles
no error): there it may be the neighbour.
"""
import numpy as np
import pytest
import torch

from hybrid_upcycling_gb300 import AdamW, State8, _lib, adamw_step, build, grad_norm
from oracle import ops_oracle as oo

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HYPER = dict(betas=(0.9, 0.999), eps=1e-8, lr=1e-3, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def cut(x, shift):
    """A copy of x that starts `shift` elements behind an allocation's start."""
    buf = torch.empty(x.numel() + shift, dtype=x.dtype, device=x.device)
    buf[shift:] = x.reshape(-1)
    return buf[shift:]


def encoded(x, seed, keep):
    q, e = oo.round_code(f64(x), oo.random_bits(seed, 0, x.numel()) & np.uint64(0xFFFF), keep)
    return State8(torch.tensor(q, dtype=torch.float32).to(torch.float8_e4m3fn).cuda(),
                  torch.tensor(e.astype(np.int8)).cuda())


def model(sizes, param, grad, bits, seed=0, shift=0):
    gen = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda n, s: torch.randn(n, generator=gen, device="cuda") * s  # noqa: E731
    w, g, m, v = [], [], [], []
    for i, n in enumerate(sizes):
        w.append(cut(rnd(n, 0.05), shift))
        g.append(cut(rnd(n, 1e-2 * 4 ** (i % 3)).to(grad), shift))
        a, r = rnd(n, 2e-3), rnd(n, 4e-3).abs() + 1e-5
        if bits == 32:
            m.append(cut(a, shift))
            v.append(cut(r * r, shift))
        else:
            m.append(encoded(a, i, False))
            v.append(encoded(r, 100 + i, True))
            if shift:
                m[-1], v[-1] = (State8(cut(s.codes.view(torch.uint8), shift), s.exponents) for s in (m[-1], v[-1]))
    p = [cut(x.bfloat16() if param != "fp32" else x, shift) for x in w]
    return p, g, m, v, w if param == "master" else None


def values(s):
    return f64(s.values()) if isinstance(s, State8) else f64(s)


def check_codes(state, x, bits16, keep):
    """The state's codes against the oracle's rounding of the exact value x."""
    if len(x) == 0:
        return
    r, step, e = oo.code_parts(x)
    q, _ = oo.round_code(x, bits16, keep)
    got = f64(state.codes.view(torch.float8_e4m3fn) if state.codes.dtype == torch.uint8 else state.codes)
    assert np.array_equal(f64(state.exponents), e)
    t = r + bits16 / 65536
    edge = np.abs(t - np.round(t)) < 1e-4
    assert np.array_equal(got[~edge], q[~edge])
    assert np.all(np.abs(got - q) <= 2.001 * step)
    assert edge.sum() <= 0.02 * len(x) + 3  # few enough that the equality above says something


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param", ["fp32", "master", "bf16"])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,shift", [([1], 0), ([255, 256, 257, 0, 3, 8], 0), ([5000, 2048, 77], 1), ([70001], 0),
                                         ([40] * 70, 0)])
def test_parity(sizes, shift, param, grad, bits):
    step, seed = 7, 3
    p, g, m, v, w = model(sizes, param, grad, bits, seed=len(sizes), shift=shift)
    before = [(f64(w[i] if w else p[i]), f64(g[i]), values(m[i]), values(v[i])) for i in range(len(sizes))]
    norm = grad_norm(g)
    ref_norm = np.sqrt(sum((b[1] ** 2).sum() for b in before))
    assert abs(norm.item() - ref_norm) <= 64 * U * ref_norm
    max_norm = 0.5 * ref_norm
    adamw_step(p, g, m, v, step=step, masters=w, norm=norm, max_norm=max_norm, seed=seed, **HYPER)
    clip = min(1.0, max_norm / (ref_norm + 1e-6))
    pos = 0
    for i, n in enumerate(sizes):
        w0, g0, m0, v0 = before[i]
        v0 = v0 ** 2 if bits == 8 else v0
        rw, rm, rv = oo.adamw(w0, g0, m0, v0, step=step, clip=clip, **HYPER)
        random = oo.random_bits(seed, pos, n)
        pos += -(-n // 256) * 256
        upd = np.abs(rw - w0 * (1 - 1e-4))
        tol = 4 * U * np.abs(w0) + 200 * U * upd
        if param == "fp32":
            assert np.all(np.abs(f64(p[i]) - rw) <= tol)
        elif param == "master":
            assert np.all(np.abs(f64(w[i]) - rw) <= tol)
            assert torch.equal(p[i], w[i].bfloat16())
        else:  # the multiple of the bf16 step at or below |w| / step + random, or its neighbour where that is close
            ulp = np.exp2(np.floor(np.log2(np.maximum(np.abs(rw), 1e-30))) - 7)
            t = np.abs(rw) / ulp + ((random * np.uint64(0x9E3779B1)) & np.uint64(0xFFFFFFFF)) // np.uint64(65536) / 65536
            edge = np.abs(t - np.round(t)) * ulp <= tol + 2 ** -15 * ulp
            want = np.floor(t) * ulp * np.sign(rw)
            assert np.array_equal(f64(p[i])[~edge], want[~edge]) and edge.sum() <= 0.05 * n + 3
            assert np.all(np.abs(f64(p[i]) - want) <= 2.001 * ulp)
        if bits == 32:
            assert np.all(np.abs(f64(m[i]) - rm) <= 80 * U * (np.abs(0.9 * m0) + np.abs(0.1 * g0 * clip)))
            assert np.all(np.abs(f64(v[i]) - rv) <= 160 * U * rv)
        else:
            check_codes(m[i], rm, random & np.uint64(0xFFFF), False)
            check_codes(v[i], np.sqrt(rv), random >> np.uint64(16), True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [0, 5], [3, 1000003, 0, 17], [9] * 1500, [50_000_000]])
def test_grad_norm(dtype, sizes):
    gen = torch.Generator("cuda").manual_seed(1)
    g = [cut(torch.randn(n, generator=gen, device="cuda").to(dtype), i % 3) for i, n in enumerate(sizes)]
    a, b = grad_norm(g), grad_norm(g)
    ref = float(torch.stack([x.double().square().sum() for x in g]).sum().sqrt())
    # a thread adds n / (152 * 8 * 256 * 4) squares per running sum, a block 256 of them
    assert abs(a.item() - ref) <= (max(sizes) / 1e6 + 64) * U * ref
    assert torch.equal(a, b)


def test_more_tensors_than_one_launch_takes():
    """700 tensors are those of one flat tensor (fp32, 32-bit states: nothing depends on the list)."""
    n = 700 * 5
    flat, g, m, v, _ = model([n], "fp32", torch.float32, 32)
    parts = [[t.clone().view(700, 5)[i] for i in range(700)] for t in (flat[0], g[0], m[0], v[0])]
    norm, many = grad_norm(g), grad_norm(parts[1])
    assert abs(norm.item() - many.item()) <= 64 * U * norm.item()
    adamw_step(flat, g, m, v, step=4, norm=norm, max_norm=0.1, **HYPER)
    adamw_step(*parts, step=4, norm=norm, max_norm=0.1, **HYPER)
    for whole, pieces in zip((flat, g, m, v), parts):
        assert torch.equal(whole[0], torch.cat(pieces))


def test_elements_and_positions_behind_2_to_32():
    """One bf16 tensor with 8-bit states of 2^32 + 700 elements: its last blocks against the oracle."""
    n, tail = (1 << 32) + 700, 700
    p = [torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    g = [torch.zeros(n, dtype=torch.bfloat16, device="cuda")]
    m, v = [State8.zeros_like(p[0])], [State8.zeros_like(p[0])]
    p[0][-tail:] = torch.randn(tail, device="cuda").bfloat16()
    g[0][-tail:] = torch.randn(tail, device="cuda").bfloat16()
    w0, g0 = f64(p[0][-tail:]), f64(g[0][-tail:])
    norm = grad_norm(g)
    assert abs(norm.item() - np.linalg.norm(g0)) <= 64 * U * np.linalg.norm(g0)
    adamw_step(p, g, m, v, step=1, seed=9, **HYPER)
    rw, rm, rv = oo.adamw(w0, g0, np.zeros(tail), np.zeros(tail), step=1, **HYPER)
    random = oo.random_bits(9, 1 << 32, tail)
    at = lambda s: State8(s.codes.view(torch.uint8)[-tail:].clone(), s.exponents[-3:].clone())  # noqa: E731
    check_codes(at(m[0]), rm, random & np.uint64(0xFFFF), False)
    check_codes(at(v[0]), np.sqrt(rv), random >> np.uint64(16), True)
    ulp = np.exp2(np.floor(np.log2(np.abs(rw))) - 7)
    assert np.all(np.abs(f64(p[0][-tail:]) - rw) <= 1.001 * ulp)
    assert torch.all(p[0][: 1 << 20] == 0) and torch.all(p[0][(1 << 31) - 500: (1 << 31) + 500] == 0)


def test_norm_of_no_elements_and_of_nan():
    z = torch.zeros(0, device="cuda")
    assert grad_norm([z]).item() == 0.0
    assert np.isnan(grad_norm([torch.tensor([1.0, float("nan")], device="cuda")]).item())
    assert np.isinf(grad_norm([torch.tensor([1.0, float("inf")], device="cuda")]).item())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_norm_that_is_not_finite_skips_the_step(bits, bad):
    p, g, m, v, w = model([1000, 3], "master", torch.float32, bits)
    g[0][5] = bad
    keep = [x.clone() for x in (*p, *w)] + [values(s) for s in (*m, *v)]
    adamw_step(p, g, m, v, step=1, masters=w, norm=grad_norm(g), max_norm=1.0, **HYPER)
    now = [*p, *w] + [values(s) for s in (*m, *v)]
    for a, b in zip(keep, now):
        assert torch.equal(a, b) if isinstance(a, torch.Tensor) else np.array_equal(a, b)


def test_8bit_states_of_values_that_are_not_finite():
    """Without a norm nothing guards the states: what is not finite becomes NaN, in its own element only (an infinite
    gradient takes its block's scale with it), and bf16 parameters follow."""
    n = 600
    for bad in (float("nan"), float("inf"), -float("inf")):
        p, g, m, v, _ = model([n], "bf16", torch.float32, 8)
        g[0][300] = bad
        adamw_step(p, g, m, v, step=3, seed=1, **HYPER)
        for s in (m[0], v[0]):
            assert torch.isnan(s.values()[300]) and torch.isfinite(s.values()).sum() == n - 1
        assert not torch.isfinite(p[0][300]) and torch.isfinite(p[0]).sum() == n - 1


def test_scale_and_clip_do_what_they_say():
    """grad_scale s with gradients g is the step with gradients s g; a norm under max_norm clips nothing."""
    p, g, m, v, _ = model([3000], "fp32", torch.float32, 32)
    q, h, mm, vv, _ = model([3000], "fp32", torch.float32, 32)
    adamw_step(p, g, m, v, step=2, grad_scale=0.25, norm=grad_norm(g), max_norm=1e9, **HYPER)
    adamw_step(q, [x * 0.25 for x in h], mm, vv, step=2, **HYPER)
    assert torch.equal(p[0], q[0]) and torch.equal(m[0], mm[0]) and torch.equal(v[0], vv[0])


def test_groups_take_their_own_lr_and_decay():
    p, g, m, v, _ = model([300, 300], "fp32", torch.float32, 32)
    old = [x.clone() for x in p]
    adamw_step(p, g, m, v, step=1, lr=[0.0, 1e-2], weight_decay=[0.5, 0.0])
    assert torch.equal(p[0], old[0]) and not torch.equal(p[1], old[1])


def test_8bit_codes_follow_small_steady_changes():
    """v decays by 0.1% a step; rounded to nearest its codes would never move. Rounded stochastically the mean of r
    over many elements follows sqrt(0.999^t) within five standard errors."""
    n, steps = 65536, 200
    p, g = [torch.zeros(n, device="cuda")], [torch.zeros(n, device="cuda")]
    m, v = [State8.zeros_like(p[0])], [State8.zeros_like(p[0])]
    v[0].codes.view(torch.uint8).fill_(0x70)  # 128
    v[0].exponents.fill_(-10)
    r0 = v[0].values().mean().item()
    for t in range(1, steps + 1):
        adamw_step(p, g, m, v, step=t, lr=0.0, seed=t)
    r = f64(v[0].values())
    # each step adds an error of at most half a step (2^-4 of the value) to an element
    err = 5 * r0 * 2.0 ** -4 * np.sqrt(steps) / np.sqrt(n) + 1e-3 * r0
    assert abs(r.mean() - r0 * 0.999 ** (steps / 2)) < err, (r.mean(), r0 * 0.999 ** (steps / 2), err)


def test_bf16_without_master_moves_by_less_than_a_step():
    n = 65536
    p, g = [torch.ones(n, dtype=torch.bfloat16, device="cuda")], [torch.ones(n, device="cuda")]
    m, v = ([torch.zeros(n, device="cuda")] for _ in range(2))
    adamw_step(p, g, m, v, step=1, lr=1e-4, weight_decay=0.0, seed=5)  # the update is 1e-4, half an ulp is 2e-3
    mean = f64(p[0]).mean()
    assert abs(mean - (1 - 1e-4)) < 5 * 2.0 ** -8 * np.sqrt(1e-4 * 256 / n)


def test_optimizer_class_state_and_streams():
    """AdamW over groups: equal to the operator by hand; its state comes back from state_dict; on another stream."""
    torch.manual_seed(0)
    mk = lambda: [torch.randn(300, 7, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).bfloat16()  # noqa: E731
                  .requires_grad_() for i in range(3)]
    for bits in (32, 8):
        a, b = mk(), mk()
        oa = AdamW([{"params": a[:2], "lr": 1e-2}, {"params": a[2:], "weight_decay": 0.0}], state_bits=bits, max_norm=1.0)
        ob = AdamW([{"params": b[:2], "lr": 1e-2}, {"params": b[2:], "weight_decay": 0.0}], state_bits=bits, max_norm=1.0)
        s = torch.cuda.Stream()
        for t in range(4):
            for x, y in zip(a, b):
                x.grad = torch.randn(300, 7, device="cuda").bfloat16()
                y.grad = x.grad.clone()
            oa.step()
            if t == 2:  # a fresh optimizer takes over from the saved state
                saved = ob.state_dict()
                ob = AdamW([{"params": b[:2], "lr": 1e-2}, {"params": b[2:], "weight_decay": 0.0}], state_bits=bits,
                           max_norm=1.0)
                ob.load_state_dict(saved)
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                ob.step()
            torch.cuda.current_stream().wait_stream(s)
            for x, y in zip(a, b):
                assert torch.equal(x, y)
        assert oa.last_norm.item() > 0
    with pytest.raises(ValueError):
        ob.load_state_dict(AdamW(mk(), state_bits=32).state_dict())


def test_a_step_is_an_in_place_operation_and_counts_when_it_ran():
    p = torch.ones(300, device="cuda", requires_grad=True)
    opt = AdamW([p])
    loss = (p * p).sum()
    opt.step([torch.ones(300, device="cuda")])
    assert opt.steps == 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with pytest.raises(ValueError):
        opt.step([torch.ones(301, device="cuda")])
    assert opt.steps == 1
    with torch.inference_mode():
        q = torch.ones(300, device="cuda")
        AdamW([q]).step([torch.ones(300, device="cuda")])
        assert torch.all(q < 1)


def test_mismatched_lists_are_refused():
    p, g, m, v, _ = model([300, 20], "fp32", torch.float32, 32)
    for bad in (lambda: adamw_step(p, g[:1], m, v, step=1, lr=0.1), lambda: adamw_step(p, g[::-1], m, v, step=1, lr=0.1),
                lambda: adamw_step(p, g, [x.bfloat16() for x in m], v, step=1, lr=0.1),
                lambda: adamw_step(p, g, m, v, step=1, lr=[0.1]), lambda: adamw_step(p, g, m, v, step=1, lr=0.1, masters=p),
                lambda: adamw_step(p, g, [State8.zeros_like(x) for x in p], v, step=1, lr=0.1),
                lambda: adamw_step([x.t() for x in (torch.zeros(4, 5, device="cuda"),)], [torch.zeros(20, device="cuda")],
                                   [torch.zeros(20, device="cuda")], [torch.zeros(20, device="cuda")], step=1, lr=0.1),
                lambda: adamw_step(p, g, m, v, step=1, lr=0.1, norm=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(_lib.HyloError):
        adamw_step(p, g, m, v, step=0, lr=0.1)


@pytest.mark.parametrize("bits,masters", [(8, False), (32, True)])
def test_the_example_learns(bits, masters):
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_head.py")
    spec = importlib.util.spec_from_file_location("train_head", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, before, after, top = ex.train(steps=12, tokens=300, hidden=64, vocab=1000, state_bits=bits, masters=masters)
    assert all(np.isfinite(losses)) and losses[-1] < losses[0] - 0.5 and after > before + 0.5
    assert top.top_tokens.shape == (4, 5) and torch.all(top.top_logprobs[:, :-1] >= top.top_logprobs[:, 1:])
