"""Layer norm, RMS norm, orthogonalised updates and the Muon step as a user calls them, beside plain torch forms of the same.

Three families of cases:
  norm   layer norm or RMS norm of the rows of a residual stream, with the sum of the stream and a branch in the same
         call or without, forward ("train" false) or with the gradients of everything;
  orth   matrices orthogonalised by five Newton-Schulz steps;
  muon   one Muon step over a list of matrices: momentum, orthogonalised update, weight decay.
"""
import math

import torch

own = False  # True: run() calls the framework's operators; False: their plain forms

DEVICE = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
STEPS, ABC, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7

# the matrices of one layer of the 1B student
LAYER = "2048x2048,512x2048,512x2048,2048x2048,8192x2048,8192x2048,2048x8192"


def listed():
    return [
        # one new token before the 8B teacher's LM head: latency
        {"name": "norm_one", "op": "norm", "rms": True, "N": 1, "d": 4096, "pad": 0, "dtype": "bf16", "weight": "same",
         "bias": False, "residual": True, "train": False},
        # a short ragged batch of a small model, rows cut out of wider ones
        {"name": "norm_odd", "op": "norm", "rms": False, "N": 1501, "d": 1001, "pad": 23, "dtype": "fp16",
         "weight": "fp32", "bias": True, "residual": False, "train": False},
        # an 8K prompt through the teacher's last norm
        {"name": "norm_prompt", "op": "norm", "rms": True, "N": 8192, "d": 4096, "pad": 0, "dtype": "bf16",
         "weight": "same", "bias": False, "residual": True, "train": False},
        # a small model's training step in fp32
        {"name": "norm_train_small", "op": "norm", "rms": False, "N": 333, "d": 520, "pad": 0, "dtype": "fp32",
         "weight": "same", "bias": True, "residual": False, "train": True},
        # the 1B student's last norm over 64K tokens, gain kept in fp32
        {"name": "norm_train_64k", "op": "norm", "rms": True, "N": 65536, "d": 2048, "pad": 0, "dtype": "bf16",
         "weight": "fp32", "bias": False, "residual": True, "train": True},
        # layer norm with gain and bias on very wide rows
        {"name": "norm_train_wide", "op": "norm", "rms": False, "N": 4096, "d": 16384, "pad": 0, "dtype": "bf16",
         "weight": "same", "bias": True, "residual": False, "train": True},
        # a small model's matrices, odd sizes, one a single row: latency
        {"name": "orth_small", "op": "orth", "shapes": "64x64,128x520,520x128,77x300,1x257,256x256", "pad": 0,
         "dtype": "fp32", "out": "bf16"},
        # one projection of the 1B student
        {"name": "orth_one", "op": "orth", "shapes": "2048x2048", "pad": 0, "dtype": "bf16", "out": "bf16"},
        # tall and odd matrices cut out of wider ones
        {"name": "orth_odd", "op": "orth", "shapes": "5003x520,1000x1001,8192x2048", "pad": 5, "dtype": "fp32",
         "out": "fp16"},
        # a small model in fp32
        {"name": "muon_small", "op": "muon", "shapes": "520x520,128x520,128x520,520x520,2048x520,2048x520,520x2048",
         "param": "fp32", "grad": "fp32"},
        # two layers of the 1B student where memory is short: bf16 weights alone
        {"name": "muon_bf16", "op": "muon", "shapes": ",".join([LAYER] * 2), "param": "bf16", "grad": "bf16"},
        # three of its layers: bf16 weights with fp32 masters, fp32 gradients
        {"name": "muon_master", "op": "muon", "shapes": ",".join([LAYER] * 3), "param": "bf16_master", "grad": "fp32"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "orth", "muon"])
    if op == "norm":
        d = _log(rng, 8, 16384)
        N = _log(rng, 1, 130_000_000 // d if d > 1900 else 70000)
        rms = rng.random() < 0.5
        dtype = rng.choice(sorted(DTYPES))
        return {"op": op, "rms": rms, "N": N, "d": d, "pad": rng.choice([0, 0, 1, 8, 100]), "dtype": dtype,
                "weight": rng.choice(["none", "same", "fp32"]), "bias": not rms and rng.random() < 0.6,
                "residual": rng.random() < 0.4, "train": rng.random() < 0.6}
    kinds = [(_log(rng, 1, 8192), _log(rng, 24, 8192)) for _ in range(rng.randint(1, 3))]
    shapes, spent = [], 0
    for _ in range(_log(rng, 1, 20)):
        rows, cols = rng.choice(kinds)
        cost = _flops(rows, cols) + 40_000 * rows * cols
        if shapes and spent + cost > 3e12:
            break
        spent += cost
        shapes.append("%dx%d" % (rows, cols))
    case = {"op": op, "shapes": ",".join(shapes)}
    if op == "orth":
        return dict(case, pad=rng.choice([0, 0, 1, 8]), dtype=rng.choice(sorted(DTYPES)), out=rng.choice(["bf16", "fp16"]))
    return dict(case, param=rng.choice(["fp32", "bf16_master", "bf16"]), grad=rng.choice(["fp32", "bf16"]))


def _shapes(case):
    return [tuple(map(int, s.split("x"))) for s in case["shapes"].split(",")]


def _flops(rows, cols):
    """Of the five steps: X X^T and A^2 are symmetric, half of their products are enough."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (3 * m * m * n + m ** 3)


def work(case):
    if case["op"] == "norm":
        n, e = case["N"] * case["d"], BYTES[case["dtype"]]
        forward, backward = (4 if case["residual"] else 2), (4 if case["residual"] else 3)
        # with gradients: s is written by the forward and read by the backward; both inputs have one gradient
        return {"bytes": n * e * (forward + (backward if case["train"] else 0)) + 8 * case["d"],
                "flops": n * (24 if case["train"] else 8)}
    elements = sum(r * c for r, c in _shapes(case))
    flops = sum(_flops(r, c) for r, c in _shapes(case))
    if case["op"] == "orth":
        return {"bytes": elements * (BYTES[case["dtype"]] + BYTES[case["out"]]), "flops": flops}
    each = {"fp32": 8, "bf16": 4, "bf16_master": 10}[case["param"]] + BYTES[case["grad"]] + 8
    return {"bytes": elements * each, "flops": flops}


def _randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEVICE) * std


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(2_000_003 + int(seed))
    return {"norm": _prepare_norm, "orth": _prepare_orth, "muon": _prepare_muon}[case["op"]](case, gen)


def _rows(gen, case, std):
    """[N, d] rows of a buffer whose rows are `pad` wider."""
    N, d, pad = case["N"], case["d"], case["pad"]
    buf = torch.empty(N, d + pad, dtype=DTYPES[case["dtype"]], device=DEVICE)
    buf[:, d:] = 50.0
    buf[:, :d] = _randn(gen, N, d) * std
    return buf[:, :d]


def _prepare_norm(case, gen):
    """A residual stream: channels of different size, some of them large, rows of different size, a mean."""
    N, d = case["N"], case["d"]
    channel = torch.exp(_randn(gen, d, std=0.3))
    channel[torch.rand(d, generator=gen, device=DEVICE) < 0.01] *= 20
    s = {"case": case, "eps": 1e-6 if case["rms"] else 1e-5}
    s["x"] = _rows(gen, case, channel * torch.exp(_randn(gen, N, 1, std=0.5))) + (0.0 if case["rms"] else 0.5)
    if case["pad"]:
        wide = torch.full((N, d + case["pad"]), 50.0, dtype=DTYPES[case["dtype"]], device=DEVICE)
        wide[:, :d] = s["x"]
        s["x"] = wide[:, :d]
    s["residual"] = _rows(gen, case, 0.5 * channel) if case["residual"] else None
    wdtype = DTYPES[case["dtype"] if case["weight"] == "same" else "fp32"]
    s["weight"] = (1 + _randn(gen, d, std=0.1)).to(wdtype) if case["weight"] != "none" else None
    s["bias"] = _randn(gen, d, std=0.1).to(wdtype) if case["bias"] else None
    if case["train"]:
        s["dy"] = _rows(gen, dict(case, pad=0), 1.0 / N)
        s["ds"] = _rows(gen, dict(case, pad=0), 1.0 / N) if case["residual"] else None
        for k in ("x", "residual", "weight", "bias"):
            if s[k] is not None:
                s[k] = s[k].detach().requires_grad_()
    return s


def _gradient(gen, rows, cols):
    """A gradient as training gives: a few strong directions and noise."""
    rank = max(1, min(rows, cols) // 16)
    strong = _randn(gen, rows, rank) * torch.logspace(0, -1.5, rank, device=DEVICE) @ _randn(gen, rank, cols)
    return strong * (1e-3 / math.sqrt(rank)) + _randn(gen, rows, cols, std=3e-4)


def _prepare_orth(case, gen):
    mats = []
    for rows, cols in _shapes(case):
        buf = torch.full((rows, cols + case["pad"]), 50.0, dtype=DTYPES[case["dtype"]], device=DEVICE)
        buf[:, :cols] = _gradient(gen, rows, cols)
        mats.append(buf[:, :cols])
    return {"case": case, "mats": mats}


def _prepare_muon(case, gen):
    """Matrices in the middle of training."""
    s = {"case": case, "p": [], "master": [], "grad": [], "m": [], "lr": 3e-4, "momentum": 0.95, "wd": 0.1, "seed": 20,
         "t": 0}
    for rows, cols in _shapes(case):
        w = _randn(gen, rows, cols, std=0.02)
        s["p"].append(w if case["param"] == "fp32" else w.bfloat16())
        s["master"].append(w)
        s["grad"].append(_gradient(gen, rows, cols).to(DTYPES[case["grad"]]))
        s["m"].append(_gradient(gen, rows, cols) * 0.4)
    if case["param"] != "bf16_master":
        s["master"] = None
    return s


def run(s):
    return {"norm": _run_norm, "orth": _run_orth, "muon": _run_muon}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------------- norms


def _run_norm(s):
    c = s["case"]
    if own:
        from hybrid_upcycling_gb300 import layer_norm, rms_norm
        if c["rms"]:
            y = rms_norm(s["x"], s["weight"], eps=s["eps"], residual=s["residual"])
        else:
            y = layer_norm(s["x"], s["weight"], s["bias"], eps=s["eps"], residual=s["residual"])
        y, total = y if c["residual"] else (y, None)
        out = {"y": y, "sum": total}
        if c["train"]:
            names = [k for k in ("x", "residual", "weight", "bias") if s[k] is not None]
            results, upstream = ((y, total), (s["dy"], s["ds"])) if c["residual"] else ((y,), (s["dy"],))
            grads = torch.autograd.grad(results, [s[k] for k in names], upstream)
            out.update(("d" + k, g) for k, g in zip(names, grads))
        return {k: v for k, v in out.items() if v is not None}
    with torch.no_grad():
        return _plain_norm(s)


def _plain_norm(s):
    c, dtype = s["case"], s["x"].dtype
    x, out = s["x"].float(), {}
    if c["residual"]:
        out["sum"] = (x + s["residual"].float()).to(dtype)
        x = out["sum"].float()
    if not c["rms"]:
        x = x - x.mean(1, keepdim=True)
    r = 1 / (x.square().mean(1, keepdim=True) + s["eps"]).sqrt()
    xh = x * r
    y = xh if s["weight"] is None else xh * s["weight"].float()
    out["y"] = (y if s["bias"] is None else y + s["bias"].float()).to(dtype)
    if c["train"]:
        dy = s["dy"].float()
        g = dy if s["weight"] is None else dy * s["weight"].float()
        dx = g - xh * (g * xh).mean(1, keepdim=True)
        if not c["rms"]:
            dx = dx - g.mean(1, keepdim=True)
        dx = dx * r
        if c["residual"]:
            dx = dx + s["ds"].float()
            out["dresidual"] = dx.to(dtype)
        out["dx"] = dx.to(dtype)
        if s["weight"] is not None:
            out["dweight"] = (dy * xh).sum(0).to(s["weight"].dtype)
        if s["bias"] is not None:
            out["dbias"] = dy.sum(0).to(s["bias"].dtype)
    return out


# --------------------------------------------------------------------------------- orthogonalised updates and Muon


def _run_orth(s):
    c = s["case"]
    if own:
        from hybrid_upcycling_gb300 import orthogonalize
        return orthogonalize(s["mats"], dtype=DTYPES[c["out"]])
    return [_orthogonal(x.float()).to(DTYPES[c["out"]]) for x in s["mats"]]


def _orthogonal(x):
    x = x / (x.square().sum().sqrt() + EPS)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.T
    a, b, c = ABC
    for _ in range(STEPS):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if tall else x


def _run_muon(s):
    c = s["case"]
    s["t"] += 1
    if own:
        from hybrid_upcycling_gb300 import muon_step
        muon_step(s["p"], s["grad"], s["m"], lr=s["lr"], momentum=s["momentum"], nesterov=True, weight_decay=s["wd"],
                  adjust="rms", masters=s["master"], seed=s["seed"] + s["t"])
    else:
        at = 0
        for i, p in enumerate(s["p"]):
            _muon(s, i, p, at)
            at += -(-p.numel() // 256) * 256
    out = {"p": s["p"], "m": s["m"]}
    return dict(out, master=s["master"]) if s["master"] else out


def _muon(s, i, p, at):
    mu, g = s["momentum"], s["grad"][i].float()
    m = mu * s["m"][i] + (1 - mu) * g
    o = _orthogonal(mu * m + (1 - mu) * g)
    w = s["master"][i] if s["master"] else p.float()
    w = w * (1 - s["lr"] * s["wd"]) - s["lr"] * 0.2 * math.sqrt(max(p.shape)) * o
    s["m"][i].copy_(m)
    if s["master"]:
        s["master"][i].copy_(w)
    elif p.dtype == torch.bfloat16:  # rounded up with the probability of the part cut off
        w = w.contiguous()
        random = _random(s["seed"] + s["t"], at, p.numel()).view(p.shape)
        w = ((w.view(torch.int32) + random.int()) & -65536).view(torch.float32)
    p.copy_(w)


def _mix(x):
    """The 32-bit finaliser of MurmurHash3 on whole numbers held in 64 bits."""
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(seed, at, n):
    """16 random bits for each of n positions of the list of weights (below 2^32), from `at` on."""
    key = _mix((seed + 0x9E3779B9) & 0xFFFFFFFF)
    bits = _mix((torch.arange(at, at + n, device=DEVICE) + key) & 0xFFFFFFFF)
    return ((bits * 0x9E3779B1) & 0xFFFFFFFF) >> 16


# ------------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    if case["op"] != "norm" and sum(_exact_flops(r, c) for r, c in _shapes(case)) > 12e12:
        return None
    s = prepare(case, seed)
    return {"norm": _exact_norm, "orth": _exact_orth, "muon": _exact_muon}[case["op"]](s)


def _exact_norm(s):
    """The definition in 64 bits on slices of rows; gradients by torch's own differentiation."""
    c, dtype = s["case"], s["x"].dtype
    names = [k for k in ("weight", "bias") if s[k] is not None]
    leaves = {k: s[k].detach().double().requires_grad_() for k in names}
    parts, sums = {}, {}
    for lo in range(0, c["N"], 4096):
        cut = slice(lo, lo + 4096)
        x = s["x"].detach()[cut].double()
        if c["residual"]:
            x = x + s["residual"].detach()[cut].double()
            parts.setdefault("sum", []).append(x)
            x = x.to(dtype).double()
        x = x.detach().requires_grad_()
        centre = 0.0 if c["rms"] else x.sum(1, keepdim=True) / c["d"]
        spread = ((x - centre) ** 2).sum(1, keepdim=True) / c["d"]
        y = (x - centre) * (spread + s["eps"]) ** -0.5
        if "weight" in leaves:
            y = y * leaves["weight"]
        if "bias" in leaves:
            y = y + leaves["bias"]
        parts.setdefault("y", []).append(y.detach())
        if c["train"]:
            got = torch.autograd.grad(y, [x] + [leaves[k] for k in names], s["dy"][cut].double())
            dx = got[0] + s["ds"][cut].double() if c["residual"] else got[0]
            parts.setdefault("dx", []).append(dx)
            for k, g in zip(names, got[1:]):
                sums["d" + k] = sums.get("d" + k, 0) + g
    out = dict({k: torch.cat(v) for k, v in parts.items()}, **sums)
    if c["train"] and c["residual"]:
        out["dresidual"] = out["dx"]
    return out


def _exact_flops(rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    return 4 * m * m * n + 8 * STEPS * m ** 3


def _exact_orthogonal(x):
    """X -> Q X with Q = p(G) p(G') p(G'') ..., all polynomials in the one matrix G = X X^T."""
    x = x.double() / (torch.linalg.norm(x.double()) + EPS)
    if x.shape[0] > x.shape[1]:
        return _exact_steps(x.T).T
    return _exact_steps(x)


def _exact_steps(x):
    a, b, c = ABC
    one = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    g, q = x @ x.T, one
    for _ in range(STEPS):
        p = a * one + g @ (b * one + c * g)
        q = p @ q
        g = p @ g @ p
    return q @ x


def _exact_orth(s):
    return [_exact_orthogonal(x) for x in s["mats"]]


def _exact_muon(s):
    c, t, out, at = s["case"], s["t"] + 1, {"p": [], "m": [], "master": []}, 0
    for i, p in enumerate(s["p"]):
        g, m = s["grad"][i].double(), s["m"][i].double()
        m = m + (1 - s["momentum"]) * (g - m)
        o = _exact_orthogonal(g + s["momentum"] * (m - g))
        w = (s["master"][i] if s["master"] else p).double()
        w = w - s["lr"] * (s["wd"] * w + 0.2 * max(p.shape) ** 0.5 * o)
        out["m"].append(m)
        out["master"].append(w)
        if c["param"] == "bf16":
            step = torch.exp2(torch.floor(torch.log2(w.abs().clamp_min(2.0 ** -126))) - 7)
            u = _random(s["seed"] + t, at, p.numel()).view(p.shape)
            w = step * torch.floor(w.abs() / step + u / 65536) * torch.sign(w)
        out["p"].append(w)
        at += -(-p.numel() // 256) * 256
    if c["param"] != "bf16_master":
        del out["master"]
    return out
