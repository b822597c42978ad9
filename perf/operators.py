"""The token log-probability and AdamW operators as a user calls them, beside plain torch forms of the same.

Three families of cases:
  logits   log-probabilities of given tokens with entropy and top alternatives from logits [N, V]
           ("score"), or the same without alternatives and with the gradient of the logits ("train");
  head     the same log-probabilities and entropy straight from hidden states [N, d] and an LM head
           [V, d] ("score"), or with the gradients of both ("train");
  adamw    one AdamW step over a list of tensors, clipped by their global gradient norm, with
           states in 32 bits or as 8-bit block-scaled codes.
"""
import math

import torch

own = False  # True: run() calls the framework's operators; False: their plain forms

DEVICE = "cuda"
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
BLOCK = 256  # elements that share one scale of an 8-bit state
BETAS, EPS = (0.9, 0.999), 1e-8


def listed():
    return [
        # one new token of a decoder whose top 20 alternatives go into the answer: latency
        {"name": "score_one", "op": "logits", "N": 1, "V": 128256, "pad": 0, "dtype": "bf16", "tau": 1.0, "k": 20,
         "mask": False, "train": False},
        # one decoding step of 48 requests under grammar masks (some leave a handful of words, one leaves none),
        # fp32 logits in rows padded to the LM head's multiple of 128 words
        {"name": "score_step", "op": "logits", "N": 48, "V": 151936, "pad": 64, "dtype": "fp32", "tau": 0.7, "k": 8,
         "mask": True, "train": False},
        # a teacher's log-probabilities and alternatives over an 8K sequence, recorded for later distillation
        {"name": "score_prompt", "op": "logits", "N": 8192, "V": 128256, "pad": 0, "dtype": "bf16", "tau": 1.0,
         "k": 16, "mask": False, "train": False},
        # a small odd vocabulary in fp16, rows at every alignment, padding tokens ignored
        {"name": "train_odd", "op": "logits", "N": 1500, "V": 33001, "pad": 0, "dtype": "fp16", "tau": 1.0, "k": 0,
         "mask": False, "train": True},
        # policy or cross-entropy loss on the logits of an 8K sequence
        {"name": "train_8k", "op": "logits", "N": 8192, "V": 128256, "pad": 0, "dtype": "bf16", "tau": 1.0, "k": 0,
         "mask": False, "train": True},
        # scoring one token with the 8B teacher's LM head: the head's bytes are the cost
        {"name": "head_one", "op": "head", "N": 1, "d": 4096, "V": 128256, "tau": 1.0, "train": False},
        # scoring an 8K sequence with the 1B student's head
        {"name": "head_prompt", "op": "head", "N": 8192, "d": 2048, "V": 128256, "tau": 1.0, "train": False},
        # a short ragged batch on a small model
        {"name": "head_train_small", "op": "head", "N": 333, "d": 520, "V": 5003, "tau": 2.0, "train": True},
        # one token chunk of the 1B student's training step
        {"name": "head_train_4k", "op": "head", "N": 4096, "d": 2048, "V": 128256, "tau": 1.0, "train": True},
        # the norm gains and biases of a small model, fp32 throughout: latency
        {"name": "adamw_small", "op": "adamw", "sizes": "2048,2048,64,1,8192,4099,2048,520,2048,128,77,2048",
         "param": "fp32", "grad": "fp32", "bits": 32},
        # the 1B student's LM head and eight of its layers' matrices: bf16 weights with fp32 masters, fp32 gradients
        {"name": "adamw_master", "op": "adamw",
         "sizes": ",".join(["262668288"] + ["4194304,1048576,1048576,4194304,16777216,16777216,16777216,2048,2048"] * 2),
         "param": "bf16_master", "grad": "fp32", "bits": 32},
        # the same weights where memory is short: bf16 weights alone, bf16 gradients, 8-bit states
        {"name": "adamw_8bit", "op": "adamw",
         "sizes": ",".join(["262668288"] + ["4194304,1048576,1048576,4194304,16777216,16777216,16777216,2048,2048"] * 2),
         "param": "bf16", "grad": "bf16", "bits": 8},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logits", "logits", "head", "head", "adamw", "adamw"])
    if op == "logits":
        train = rng.random() < 0.5
        V = _log(rng, 300, 260000)
        N = _log(rng, 1, min(8192, 1_000_000_000 // V))
        return {"op": op, "N": N, "V": V, "pad": rng.choice([0, 0, 1, 64, 100]), "dtype": rng.choice(sorted(DTYPES)),
                "tau": rng.choice([0.6, 1.0, 2.0]), "k": 0 if train else rng.randint(0, 32),
                "mask": rng.random() < 0.4, "train": train}
    if op == "head":
        train = rng.random() < 0.5
        V = _log(rng, 300, 160000)
        d = 8 * _log(rng, 8, 512)
        d = 3080 if d == 3072 else d
        N = _log(rng, 1, min(8192, (1_000_000_000_000 if train else 2_000_000_000_000) // (V * d)))
        return {"op": op, "N": N, "d": d, "V": V, "tau": rng.choice([0.7, 1.0, 2.0]), "train": train}
    count, total = _log(rng, 1, 48), _log(rng, 3000, 300_000_000)
    parts = [rng.random() ** 3 + 1e-3 for _ in range(count)]
    sizes = [max(1, int(total * p / sum(parts))) for p in parts]
    return {"op": op, "sizes": ",".join(map(str, sizes)), "param": rng.choice(["fp32", "bf16_master", "bf16"]),
            "grad": rng.choice(["fp32", "bf16"]), "bits": rng.choice([8, 32])}


def _sizes(case):
    return [int(x) for x in case["sizes"].split(",")]


def _randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device=DEVICE) * std


def prepare(case, seed):
    gen = torch.Generator(DEVICE).manual_seed(1_000_003 + int(seed))
    return {"logits": _prepare_logits, "head": _prepare_head, "adamw": _prepare_adamw}[case["op"]](case, gen)


def _tokens(gen, N, V):
    tokens = torch.randint(0, V, (N,), generator=gen, device=DEVICE)
    tokens[7::29] = -100  # padding positions are ignored
    return tokens


def _prepare_logits(case, gen):
    """Logits with the spread of an LM head on normalised states, the true token raised in most rows."""
    N, V, pad, dtype = case["N"], case["V"], case["pad"], DTYPES[case["dtype"]]
    tokens = _tokens(gen, N, V)
    buf = torch.empty(N, V + pad, dtype=dtype, device=DEVICE)
    z = buf[:, :V]
    for r in range(0, N, 1024):
        z[r:r + 1024] = _randn(gen, min(1024, N - r), V, std=1.3)
    rows = torch.arange(N, device=DEVICE)
    hit = tokens.clamp_min(0)
    z[rows, hit] += (10 * torch.rand(N, generator=gen, device=DEVICE)).to(dtype)
    if case["mask"]:
        kept = z[rows, hit].clone()
        for r in range(0, N, 5):  # a grammar that leaves five words: the token and four others
            few = torch.randint(0, V, (4,), generator=gen, device=DEVICE)
            left = z[r, few].clone()
            z[r] = -math.inf
            z[r, few] = left
        for r in range(3, N, 5):  # half of the vocabulary is not allowed
            z[r, : V // 2] = -math.inf
        z[rows, hit] = kept
        z[1::24] = -math.inf  # a mask that leaves nothing
    buf[:, V:] = 50.0  # what lies in a padded row's end is not part of it
    s = {"case": case, "z": z, "tokens": tokens}
    if case["train"]:
        s["g_logp"] = -torch.rand(N, generator=gen, device=DEVICE) / N
        s["g_ent"] = _randn(gen, N, std=0.1 / N)
        s["z"] = z.detach().requires_grad_()
    return s


def _prepare_head(case, gen):
    """RMS-normalised hidden states and a head of standard deviation 0.02; tokens near the model's own choice."""
    N, d, V = case["N"], case["d"], case["V"]
    W = torch.empty(V, d, dtype=torch.bfloat16, device=DEVICE)
    for r in range(0, V, 16384):
        W[r:r + 16384] = _randn(gen, min(16384, V - r), d, std=0.02)
    tokens = _tokens(gen, N, V)
    h = _randn(gen, N, d) + 0.1 * W[tokens.clamp_min(0)].float() / 0.02
    h = (h / h.square().mean(1, keepdim=True).sqrt()).bfloat16()
    s = {"case": case, "h": h, "W": W, "tokens": tokens}
    if case["train"]:
        s["g_logp"] = -torch.rand(N, generator=gen, device=DEVICE) / N
        s["g_ent"] = _randn(gen, N, std=0.1 / N)
        h.requires_grad_()
        W.requires_grad_()
    return s


def _padded(n):
    return -(-n // BLOCK) * BLOCK


def _prepare_adamw(case, gen):
    """A model in the middle of training. Every kind of tensor lies in one buffer, each tensor from a multiple of
    256 elements on (as a trainer with gradient buckets keeps them); the gaps hold zeros."""
    sizes = _sizes(case)
    starts, total = [], 0
    for n in sizes:
        starts.append(total)
        total += _padded(n)
    real = torch.zeros(total, dtype=torch.bool, device=DEVICE)
    for a, n in zip(starts, sizes):
        real[a:a + n] = True

    def fill(std):
        return _randn(gen, total, std=std).mul_(real)

    w = fill(0.02)
    scale = torch.exp2(torch.randint(-3, 4, (total // BLOCK,), generator=gen, device=DEVICE).float())
    scale = scale.repeat_interleave(BLOCK)  # gradients differ in size from row to row
    grad = (fill(1e-3) * scale).to(DTYPES[case["grad"]])
    m = fill(3e-4) * scale
    r = fill(1e-3).abs_().mul_(scale).add_(1e-4).mul_(real)
    s = {"case": case, "sizes": sizes, "starts": starts, "total": total, "t": 100, "lr": 1e-3, "wd": 0.1,
         "max_norm": 1.0, "seed": 20, "grad": grad}
    s["p"] = w.clone() if case["param"] == "fp32" else w.bfloat16()
    if case["param"] == "bf16_master":
        s["master"] = w
    if case["bits"] == 32:
        s["m"], s["v"] = m, r.square_()
    else:
        s["m"], s["m_exp"] = _encode(m)
        s["r"], s["r_exp"] = _encode(r)
    views = {}
    for key in ("p", "grad", "master", "m", "v", "r"):
        if key in s:
            views[key] = [s[key][a:a + n] for a, n in zip(starts, sizes)]
    for key in ("m_exp", "r_exp"):
        if key in s:
            views[key] = [s[key][a // BLOCK:(a + _padded(n)) // BLOCK] for a, n in zip(starts, sizes)]
    s["views"] = views
    return s


def _encode(x):
    """x as e4m3 codes (nearest) with one power of two per block."""
    e = _block_exponent(x)
    return (x * torch.exp2(-e.float()).repeat_interleave(BLOCK)).to(torch.float8_e4m3fn), e


def _block_exponent(x):
    """The block's power of two brings its largest magnitude into [128, 256); int8, within [-120, 120]."""
    top = x.abs().view(-1, BLOCK).amax(1)
    return (torch.frexp(top)[1] - 1 - 7).where(top > 0, torch.full_like(top, -120).int()).clamp(-120, 120).to(torch.int8)


def run(s):
    return {"logits": _run_logits, "head": _run_head, "adamw": _run_adamw}[s["case"]["op"]](s)


def work(case):
    if case["op"] == "logits":
        n = case["N"] * case["V"]
        return {"bytes": n * BYTES[case["dtype"]] * (2 if case["train"] else 1) + case["N"] * (16 + 12 * case["k"]),
                "flops": n * (12 if case["train"] else 6)}
    if case["op"] == "head":
        n = case["N"] * case["V"] * case["d"]
        b = 2 * case["d"] * (case["N"] + case["V"])
        return {"bytes": b * (2 if case["train"] else 1) + 16 * case["N"], "flops": n * (6 if case["train"] else 2)}
    n = sum(_sizes(case))
    each = {"fp32": 8, "bf16": 4, "bf16_master": 10}[case["param"]] + BYTES[case["grad"]]
    each += 16 if case["bits"] == 32 else 4 + 4 / BLOCK
    return {"bytes": n * each, "flops": n * 16}


# ---------------------------------------------------------------------------------- log-probabilities of tokens


def _run_logits(s):
    c = s["case"]
    if own:
        from hybrid_upcycling_gb300 import token_logprobs
        r = token_logprobs(s["z"], s["tokens"], tau=c["tau"], top_k=c["k"])
        if c["train"]:
            dz, = torch.autograd.grad((r.logprobs, r.entropy), (s["z"],), (s["g_logp"], s["g_ent"]))
            return {"logprobs": r.logprobs, "entropy": r.entropy, "dz": dz}
        return {"logprobs": r.logprobs, "entropy": r.entropy, "top_logprobs": r.top_logprobs, "top_tokens": r.top_tokens}
    with torch.no_grad():
        z = s["z"].float()
        lp, logp, ent = _logprobs(z, s["tokens"], c["tau"])
        if c["train"]:
            dz = _logits_grad(lp, ent, s["tokens"], c["tau"], s["g_logp"], s["g_ent"])
            return {"logprobs": logp, "entropy": ent, "dz": dz.to(s["z"].dtype)}
        ids = _top(z, c["k"])
        return {"logprobs": logp, "entropy": ent, "top_logprobs": lp.gather(1, ids), "top_tokens": ids}


def _logprobs(z, tokens, tau):
    """All log-probabilities, the tokens', and the entropy. A row of -inf has log-probabilities -inf and entropy 0."""
    y = z / tau
    m = y.amax(1, keepdim=True)
    y = y - torch.where(m == -math.inf, torch.zeros_like(m), m)
    sums = y.exp().sum(1, keepdim=True)
    lp = torch.where(sums > 0, y - sums.log(), y)
    ent = -torch.where(lp == -math.inf, torch.zeros_like(lp), lp.exp() * lp).sum(1)
    logp = lp.gather(1, tokens.clamp_min(0)[:, None])[:, 0]
    return lp, torch.where(tokens < 0, torch.zeros_like(logp), logp), ent


def _logits_grad(lp, ent, tokens, tau, g_logp, g_ent):
    """d(sum g_logp logp + g_ent entropy) / dz; nothing for a row that allows nothing."""
    p = lp.exp()
    g = torch.where(tokens < 0, torch.zeros_like(g_logp), g_logp)
    dz = -p * (g[:, None] + g_ent[:, None] * torch.where(p > 0, lp + ent[:, None], torch.zeros_like(lp)))
    dz.scatter_add_(1, tokens.clamp_min(0)[:, None], g[:, None])
    return torch.where(p.sum(1, keepdim=True) > 0, dz / tau, torch.zeros_like(dz))


def _top(z, k):
    """The k largest of each row, largest first, ties to the lowest index: by one whole number per word that orders both."""
    bits = (z + 0.0).view(torch.int32).to(torch.int64)
    order = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))
    key = order * (1 << 31) + ((1 << 31) - 1 - torch.arange(z.shape[1], device=z.device))
    return key.topk(k, dim=1).indices


def _run_head(s):
    c = s["case"]
    if own:
        from hybrid_upcycling_gb300 import head_logprobs
        logp, ent = head_logprobs(s["h"], s["W"], s["tokens"], tau=c["tau"])
        if c["train"]:
            dh, dW = torch.autograd.grad((logp, ent), (s["h"], s["W"]), (s["g_logp"], s["g_ent"]))
            return {"logprobs": logp, "entropy": ent, "dh": dh, "dW": dW}
        return {"logprobs": logp, "entropy": ent}
    with torch.no_grad():
        h, W = s["h"].float(), s["W"].float()
        lp, logp, ent = _logprobs(h @ W.T, s["tokens"], c["tau"])
        if not c["train"]:
            return {"logprobs": logp, "entropy": ent}
        G = _logits_grad(lp, ent, s["tokens"], c["tau"], s["g_logp"], s["g_ent"])
        return {"logprobs": logp, "entropy": ent, "dh": (G @ W).bfloat16(), "dW": (G.T @ h).bfloat16()}


# ---------------------------------------------------------------------------------------------------- AdamW


def _run_adamw(s):
    c = s["case"]
    s["t"] += 1
    if own:
        from hybrid_upcycling_gb300 import State8, adamw_step, grad_norm
        v = s["views"]
        if c["bits"] == 32:
            m, vv = v["m"], v["v"]
        else:
            m = [State8(*x) for x in zip(v["m"], v["m_exp"])]
            vv = [State8(*x) for x in zip(v["r"], v["r_exp"])]
        norm = grad_norm(v["grad"])
        adamw_step(v["p"], v["grad"], m, vv, step=s["t"], lr=s["lr"], betas=BETAS, eps=EPS, weight_decay=s["wd"],
                   masters=v.get("master"), norm=norm, max_norm=s["max_norm"], seed=s["seed"] + s["t"])
    else:
        norm = _adamw(s)
    out = {"norm": norm, "p": s["p"]}
    for key in ("master", "m", "v", "r"):
        if key in s:
            out[key] = s[key]
    for key in ("m_exp", "r_exp"):
        if key in s:
            out[key] = s[key].bfloat16()
    return out


def _adamw(s):
    c, t, (b1, b2) = s["case"], s["t"], BETAS
    g = s["grad"].float()
    norm = g.square().sum().sqrt().view(1)
    g = g * (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    if c["bits"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = s["m"].float() * torch.exp2(s["m_exp"].float()).repeat_interleave(BLOCK)
        v = (s["r"].float() * torch.exp2(s["r_exp"].float()).repeat_interleave(BLOCK)).square()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g.square()
    p = s["master"] if c["param"] == "bf16_master" else s["p"].float()
    p = p * (1 - s["lr"] * s["wd"]) - s["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + EPS)
    random = None
    if c["bits"] == 8 or c["param"] == "bf16":
        random = _random(s["seed"] + t, s["total"])
    if c["bits"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        r = v.sqrt()
        s["m_exp"].copy_(_block_exponent(m))
        s["r_exp"].copy_(_block_exponent(r))
        s["m"].copy_(_round8(m, s["m_exp"], random & 0xFFFF, False))
        s["r"].copy_(_round8(r, s["r_exp"], random >> 16, True))
    if c["param"] == "bf16":
        p = ((p.view(torch.int32) + (((random * 0x9E3779B1) & 0xFFFFFFFF) >> 16).int()) & -65536).view(torch.float32)
    if c["param"] == "bf16_master":
        s["master"].copy_(p)
    s["p"].copy_(p)
    return norm


def _mix(x):
    """The 32-bit finaliser of MurmurHash3 on whole numbers held in 64 bits."""
    x = ((x ^ (x >> 16)) * 0x85EBCA6B) & 0xFFFFFFFF
    x = ((x ^ (x >> 13)) * 0xC2B2AE35) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random(seed, n):
    """32 random bits for each of n < 2^32 positions of the list."""
    key = _mix((seed + 0x9E3779B9) & 0xFFFFFFFF)
    return _mix((torch.arange(n, device=DEVICE) + key) & 0xFFFFFFFF)


def _round8(x, e, random, keep):
    """x 2^-e to an e4m3 value, up with the probability of the part cut off (16 random bits); `keep`: not to zero."""
    x = x * torch.exp2(-e.float()).repeat_interleave(BLOCK)
    a = x.abs()
    low = torch.where(a < 2.0 ** -6, 2.0 ** -6, 0.0)  # subnormal codes: the same steps as just above
    q = (((a + low).view(torch.int32) + (random << 4).int()) & -1048576).view(torch.float32) - low
    if keep:
        q = torch.where(a > 0, q.clamp_min(2.0 ** -9), q)
    return torch.copysign(q, x)


# ------------------------------------------------------------------------------------------- in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"logits": _exact_logits, "head": _exact_head, "adamw": _exact_adamw}[case["op"]](s)


def _exact_rows(z, s, lo, hi, grads):
    """Rows lo..hi of logits z (64 bits): softmax by torch's own, entropy by its sum, gradient by the definition."""
    tau, tok = s["case"]["tau"], s["tokens"][lo:hi]
    empty = (z == -math.inf).all(1)
    y = torch.where(empty[:, None], torch.zeros_like(z), z / tau)
    lp = torch.log_softmax(y, 1)
    p = lp.exp()
    ent = torch.special.entr(p).sum(1)
    at = lp[torch.arange(hi - lo, device=z.device), tok.clamp_min(0)]
    at[empty] = -math.inf
    at[tok < 0] = 0.0
    ent[empty] = 0.0
    lp[empty] = -math.inf
    if not grads:
        return lp, at, ent, None
    one = torch.zeros_like(p)
    one[torch.arange(hi - lo, device=z.device), tok.clamp_min(0)] = 1.0
    a = s["g_logp"][lo:hi].double() * (tok >= 0)
    b = s["g_ent"][lo:hi].double()
    d = a[:, None] * (one - p) + b[:, None] * (torch.special.entr(p) - p * ent[:, None])
    d[empty] = 0.0
    return lp, at, ent, d / tau


def _exact_logits(s):
    c, z = s["case"], s["z"].detach()
    parts = []
    for lo in range(0, c["N"], 512):
        hi = min(c["N"], lo + 512)
        x = z[lo:hi].double()
        lp, at, ent, d = _exact_rows(x, s, lo, hi, c["train"])
        if c["train"]:
            parts.append((at, ent, d))
        else:
            ids = torch.sort(x + 0.0, dim=1, descending=True, stable=True).indices[:, :c["k"]]
            parts.append((at, ent, lp.gather(1, ids), ids))
    names = ("logprobs", "entropy", "dz") if c["train"] else ("logprobs", "entropy", "top_logprobs", "top_tokens")
    return dict(zip(names, (torch.cat(x) for x in zip(*parts))))


def _exact_head(s):
    c = s["case"]
    h, W = s["h"].detach().double(), s["W"].detach().double()
    at, ent, dh = [], [], []
    dW = torch.zeros_like(W) if c["train"] else None
    for lo in range(0, c["N"], 1024):
        hi = min(c["N"], lo + 1024)
        _, a, e, d = _exact_rows(h[lo:hi] @ W.T, s, lo, hi, c["train"])
        at.append(a)
        ent.append(e)
        if c["train"]:
            dh.append(d @ W)
            dW += d.T @ h[lo:hi]
    out = {"logprobs": torch.cat(at), "entropy": torch.cat(ent)}
    return dict(out, dh=torch.cat(dh), dW=dW) if c["train"] else out


def _exact_adamw(s):
    """Tensor by tensor, with the rounding as its definition has it: the multiple of the step below |x| / step + u."""
    c, t, (b1, b2) = s["case"], s["t"] + 1, BETAS
    norm = sum((g.double() ** 2).sum() for g in s["views"]["grad"]).sqrt()
    clip = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    out = {k: torch.zeros(s["total"], dtype=torch.float64, device=DEVICE) for k in ("p", "master", "m", "v", "r")}
    out.update({k: torch.full((s["total"] // BLOCK,), -120.0, dtype=torch.float64, device=DEVICE) for k in ("m_exp", "r_exp")})
    key = _mix((s["seed"] + t + 0x9E3779B9) % (1 << 32))
    scaled = lambda q, e: q.double() * torch.exp2(e.double()).repeat_interleave(BLOCK)[:q.numel()]  # noqa: E731
    for i, (a, n) in enumerate(zip(s["starts"], s["sizes"])):
        view = {k: x[i] for k, x in s["views"].items()}
        g = view["grad"].double() * clip
        m = view["m"].double() if c["bits"] == 32 else scaled(view["m"], view["m_exp"])
        v = view["v"].double() if c["bits"] == 32 else scaled(view["r"], view["r_exp"]) ** 2
        m = m + (1 - b1) * (g - m)
        v = v + (1 - b2) * (g * g - v)
        w = view["master" if "master" in view else "p"].double()
        w = w - s["lr"] * (s["wd"] * w + m / (1 - b1 ** t) / ((v / (1 - b2 ** t)) ** 0.5 + EPS))
        bits = _mix((torch.arange(a, a + n, device=DEVICE) + key) % (1 << 32))
        if c["bits"] == 32:
            out["m"][a:a + n], out["v"][a:a + n] = m, v
        else:
            for name, x, u in (("m", m, bits % 65536), ("r", v ** 0.5, bits // 65536)):
                full = torch.zeros(_padded(n), dtype=torch.float64, device=DEVICE)
                full[:n] = x.abs()
                top = full.view(-1, BLOCK).amax(1)
                e = torch.where(top > 0, torch.floor(torch.log2(top)) - 7, -120.0).clamp(-120, 120)
                y = x.abs() * torch.exp2(-e).repeat_interleave(BLOCK)[:n]
                step = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
                q = step * torch.floor(y / step + u / 65536)
                if name == "r":
                    q = torch.where(y > 0, q.clamp_min(2.0 ** -9), q)
                out[name][a:a + n] = q * torch.sign(x)
                out[name + "_exp"][a // BLOCK:(a + _padded(n)) // BLOCK] = e
        if "master" in view:
            out["master"][a:a + n] = w
        if c["param"] == "bf16":
            step = torch.exp2(torch.floor(torch.log2(w.abs().clamp_min(2.0 ** -126))) - 7)
            u = (bits * 0x9E3779B1 % (1 << 32)) // 65536
            w = step * torch.floor(w.abs() / step + u / 65536) * torch.sign(w)
        out["p"][a:a + n] = w
    keep = ["p"] + [k for k in ("master", "m", "v", "r", "m_exp", "r_exp") if k in s]
    return dict({k: out[k] for k in keep}, norm=norm.view(1))
