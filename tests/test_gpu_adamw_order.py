"""8-bit AdamW states over consecutive steps: codes and exponents are exactly those of the documented order of rounding.

The reference is that order in elementary fp32 torch operations (each rounds to nearest by itself). Moments, codes
and exponents have no tolerance: a value that differs in its last bit falls on the other side of its random
threshold for one element in about 2^20, and the next step carries the whole code's difference into the
parameters. The parameter's own update has no documented order: per step two rounded operations of its size and 32
of the update's, u = 2^-24 each, so t steps are within 2 t u |w| + 32 t u (sum of the updates' magnitudes).
"""
import pytest
import torch

from hybrid_upcycling_gb300 import State8, _lib, adamw_step, build, grad_norm

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BLOCK = 256
B1, B2, EPS, LR, WD = 0.9, 0.999, 1e-8, 1e-3, 0.1


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    return _lib.load()


def mix(x):
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(seed, start, n):
    """32 random bits for positions start .. start + n - 1 < 2^32."""
    return mix((torch.arange(start, start + n, device="cuda") + mix((seed + 0x9E3779B9) & 0xFFFFFFFF)) & 0xFFFFFFFF)


def blocks(x):
    return torch.nn.functional.pad(x, (0, -x.numel() % BLOCK)).view(-1, BLOCK)


def exponents(x):
    top = blocks(x.abs()).amax(1)
    e = torch.frexp(top)[1] - 8
    return torch.where(top > 0, e, torch.full_like(e, -120)).clamp(-120, 120)


def spread(e, n):
    """2^e for every element, exactly."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).repeat_interleave(BLOCK)[:n]


def encode(x, bits16, keep):
    """(values of the codes before the power of two, exponents)."""
    e = exponents(x)
    y = x.abs() * spread(-e, x.numel())
    y = torch.where(y < 2.0 ** -6, (y + 2.0 ** -6) - 2.0 ** -6, y)  # to a multiple of 2^-29
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y.clamp_min(2.0 ** -6))[1] - 4)
    q = (y.double() / step + bits16.double() / 65536).floor() * step  # exact in 64 bits
    if keep:
        q = torch.where(y > 0, q.clamp_min(2.0 ** -9), q)
    return torch.copysign(q.float(), x), e


def decoded(s):
    n = s.codes.numel()
    return s.codes.float() * spread(s.exponents.int(), n)


def reference(w, g, q, qe, r, re, clip, t, seed, start):
    """One step for one tensor, each operation rounded to fp32: (w, size of the update, m's codes, r's codes)."""
    g = g.float() * clip
    m = B1 * (q * spread(qe, q.numel())) + (1 - B1) * g
    v0 = r * spread(re, r.numel())
    v = B2 * (v0 * v0) + (1 - B2) * (g * g)
    root = torch.where(v < 2.0 ** -126, 0.0, v).sqrt()
    update = LR * (m.double() / (1 - B1 ** t)) / (v.double().sqrt() / (1 - B2 ** t) ** 0.5 + EPS)
    w = (w.double() * (1 - LR * WD) - update).float()
    bits = random_bits(seed, start, w.numel())
    return w, update.abs(), encode(m, bits & 0xFFFF, False), encode(root, bits >> 16, True)


@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("param,sizes,shift", [
    ("master", [9_000_000, 3_000_001, 777, 1, 2048], 0), ("fp32", [12_000_000, 256, 255], 0), ("bf16", [11_000_003, 64], 0),
    ("master", [70_001, 4099], 1)])
def test_four_steps(param, sizes, shift, grad):
    gen = torch.Generator("cuda").manual_seed(11)
    rnd = lambda n: torch.randn(n, generator=gen, device="cuda")  # noqa: E731
    cut = lambda x: torch.cat([x[:shift], x])[shift:] if shift else x  # noqa: E731
    w, p, ms, vs, ref, starts, total = [], [], [], [], [], [], 0
    for n in sizes:
        starts.append(total)
        total += -(-n // BLOCK) * BLOCK
        scale = torch.exp2(torch.randint(-3, 4, (-(-n // BLOCK),), generator=gen, device="cuda").float())
        scale[::50] *= 2.0 ** -60  # squares that fp32 holds with few bits or none
        scale = scale.repeat_interleave(BLOCK)[:n]
        x = rnd(n) * 0.02
        m, r = rnd(n) * 3e-4 * scale, (rnd(n).abs() * 1e-3 + 1e-4) * scale
        p.append(cut(x if param == "fp32" else x.bfloat16()))
        w.append(cut(x) if param == "master" else None)
        state = []
        for y, keep in ((m, False), (r, True)):
            q, e = encode(y, torch.zeros(n, dtype=torch.int64, device="cuda"), keep)
            state.append((q, e))
            (ms if not keep else vs).append(State8(cut(q.to(torch.float8_e4m3fn).view(torch.uint8)).view(torch.float8_e4m3fn),
                                                   e.to(torch.int8)))
        ref.append([(p[-1] if param != "master" else w[-1]).float().clone(), torch.zeros(n, device="cuda", dtype=torch.float64),
                    *state, scale])
    masters = w if param == "master" else None
    seen = 0
    for t in range(101, 105):
        g = [cut((rnd(n) * 1e-3 * s[4]).to(grad)) for n, s in zip(sizes, ref)]
        norm = grad_norm(g)
        clip = (1.0 / (norm + 1e-6)).clamp(max=1.0)
        adamw_step(p, g, ms, vs, step=t, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=WD, masters=masters, norm=norm,
                   max_norm=1.0, seed=20 + t)
        for i, s in enumerate(ref):
            x, moved, m, r = reference(s[0], g[i], *s[2], *s[3], clip, t, 20 + t, starts[i])
            s[1] += moved
            s[2:4] = m, r
            for state, (q, e), name in ((ms[i], m, "m"), (vs[i], r, "r")):
                assert torch.equal(state.exponents.int(), e.int()), (t, i, name)
                wrong = (state.codes.float() != q).sum().item()
                assert wrong == 0, (t, i, name, wrong)
                seen += q.numel()
            if param == "bf16":
                s[0] = p[i].float()  # (its random rounding has a test of its own)
            else:
                s[0] = x
                got = (w if masters else p)[i]
                tol = (t - 100) * U * (2 * x.abs().double() + 32 * s[1])
                assert torch.all((got.double() - x.double()).abs() <= tol), (t, i)
                assert masters is None or torch.equal(p[i], got.bfloat16())
    assert seen == 8 * sum(sizes)
