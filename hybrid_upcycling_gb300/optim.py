"""AdamW over many tensors in one launch, with states in 32 or 8 bits, and the global gradient norm.

``grad_norm(grads)`` and ``adamw_step(params, grads, exp_avgs, exp_avg_sqs, ...)`` are the operators
(include/hylo_ops.h has the formulas); ``AdamW`` keeps the states of a list of parameters.
PyTorch only allocates memory; the step runs on the current stream and never waits for the host: the
norm that clips it stays on the device, and a step whose norm is not finite changes nothing.
"""
from __future__ import annotations

from typing import Iterable, List, NamedTuple, Optional, Sequence, Tuple, Union

import torch
from torch.autograd.graph import increment_version

from . import _lib

BLOCK = 256  # elements that share one exponent of an 8-bit state


class State8(NamedTuple):
    """A moment in 8 bits: value = code 2^exponent (for the second moment: of its square root)."""
    codes: torch.Tensor      # e4m3, torch.float8_e4m3fn or uint8, as many as the parameter's elements
    exponents: torch.Tensor  # int8 [ceil(n / 256)]

    @classmethod
    def zeros_like(cls, param: torch.Tensor) -> "State8":
        n = param.numel()
        return cls(torch.zeros(n, dtype=torch.uint8, device=param.device).view(torch.float8_e4m3fn),
                   torch.full((-(-n // BLOCK),), -120, dtype=torch.int8, device=param.device))

    def values(self) -> torch.Tensor:
        """The values the codes stand for (fp32, flat)."""
        c = self.codes.reshape(-1)
        q = (c.view(torch.float8_e4m3fn) if c.dtype == torch.uint8 else c).float()
        return q * torch.exp2(self.exponents.float()).repeat_interleave(BLOCK)[: q.numel()]


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _check_list(name: str, tensors: Sequence[torch.Tensor], dtypes, device: int, counts=None) -> None:
    for i, t in enumerate(tensors):
        if t.dtype not in dtypes or not t.is_contiguous() or t.get_device() != device:
            raise ValueError(f"{name}[{i}] must be a contiguous {' or '.join(map(str, dtypes))} tensor on the current "
                             f"CUDA device")
    if counts is not None and [t.numel() for t in tensors] != counts:
        raise ValueError(f"{name} must have the element counts {counts}")


def grad_norm(grads: Iterable[torch.Tensor]) -> torch.Tensor:
    """sqrt of the sum of squares over all gradients (fp32 or bf16, one dtype), as an fp32 tensor [1] on the device."""
    grads = list(grads)
    if not grads:
        raise ValueError("grad_norm needs at least one gradient")
    dtype = grads[0].dtype
    if dtype not in (torch.float32, torch.bfloat16) or not grads[0].is_cuda:
        raise ValueError("gradients must be float32 or bfloat16 CUDA tensors")
    _check_list("grads", grads, (dtype,), torch.cuda.current_device())
    device = grads[0].device
    norm = torch.empty(1, dtype=torch.float32, device=device)
    ws = torch.empty(_norm_workspace(), dtype=torch.uint8, device=device)
    _lib.hylo_grad_norm([g.data_ptr() for g in grads], [g.numel() for g in grads], dtype, norm, ws,
                        _lib.current_raw_stream(device.index))
    return norm


_norm_bytes = 0


def _norm_workspace() -> int:
    global _norm_bytes
    if _norm_bytes == 0:
        _norm_bytes = _lib.hylo_grad_norm_workspace_bytes()
    return _norm_bytes


def _per_tensor(x, n: int) -> Sequence[float]:
    if not isinstance(x, (list, tuple)):
        return [float(x)] * n
    if len(x) != n:
        raise ValueError("lr and weight_decay are numbers, or lists with one number per tensor")
    return x


Moments = Sequence[Union[torch.Tensor, State8]]


def adamw_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], exp_avgs: Moments, exp_avg_sqs: Moments,
               *, step: int, lr, betas: Tuple[float, float] = (0.9, 0.999), eps: float = 1e-8, weight_decay=0.0,
               masters: Optional[Sequence[torch.Tensor]] = None, norm: Optional[torch.Tensor] = None,
               max_norm: float = 1.0, grad_scale: float = 1.0, seed: int = 0) -> None:
    """One AdamW step, in place, over lists of tensors (step counts from 1). Tensors that are written may not overlap.

    params: all float32, or all bfloat16, then with fp32 ``masters`` (the step is taken on those) or without
    (the result is rounded stochastically from ``seed``: pass another one each step). grads: all
    float32 or all bfloat16. exp_avgs and exp_avg_sqs: float32 tensors, or State8 throughout (rounded
    stochastically too). lr and weight_decay: numbers, or one per tensor. grad_scale multiplies the
    gradients. norm (see grad_norm; of the gradients before grad_scale) clips them to max_norm; a norm
    that is not finite skips the step. A step cannot be captured into a CUDA graph: step, lr and seed are host values, which
    every replay would repeat (grad_norm can)."""
    params, grads = list(params), list(grads)
    n = len(params)
    if not (len(grads) == len(exp_avgs) == len(exp_avg_sqs) == n and (masters is None or len(masters) == n)):
        raise ValueError("params, grads, exp_avgs, exp_avg_sqs and masters must have the same length")
    if n == 0:
        return
    if not params[0].is_cuda:
        raise ValueError("params must be CUDA tensors")
    dev = torch.cuda.current_device()
    pdt, gdt = params[0].dtype, grads[0].dtype
    for name, dt in (("params", pdt), ("grads", gdt)):
        if dt not in (torch.float32, torch.bfloat16):
            raise ValueError(f"{name} must be float32 or bfloat16")
    if masters is not None and pdt != torch.bfloat16:
        raise ValueError("masters go with bfloat16 params")
    if norm is not None and (norm.dtype != torch.float32 or norm.numel() != 1 or norm.get_device() != dev):
        raise ValueError("norm must be one float32 value on the current CUDA device")
    bits = 8 if isinstance(exp_avgs[0], State8) else 32
    if any(isinstance(s, State8) != (bits == 8) for s in (*exp_avgs, *exp_avg_sqs)):
        raise ValueError("exp_avgs and exp_avg_sqs must be State8 throughout, or tensors throughout")
    m, v = exp_avgs, exp_avg_sqs
    sizes = [p.numel() for p in params]
    none = [0] * n
    exps = (none, none)
    lists = [("params", params, (pdt,), sizes), ("grads", grads, (gdt,), sizes)]
    if bits == 8:
        blocks = [-(-k // BLOCK) for k in sizes]
        for name, states in (("exp_avgs", m), ("exp_avg_sqs", v)):
            lists += [(name + ".codes", [s.codes for s in states], _CODES, sizes),
                      (name + ".exponents", [s.exponents for s in states], (torch.int8,), blocks)]
        exps = tuple([s.exponents.data_ptr() for s in states] for states in (m, v))
        m, v = [s.codes for s in m], [s.codes for s in v]
    else:
        lists += [("exp_avgs", m, (torch.float32,), sizes), ("exp_avg_sqs", v, (torch.float32,), sizes)]
    if masters is not None:
        lists.append(("masters", masters, (torch.float32,), sizes))
    for name, tensors, dtypes, counts in lists:
        _check_list(name, tensors, dtypes, dev, counts)
    mast = none if masters is None else [t.data_ptr() for t in masters]
    columns = ([t.data_ptr() for t in params], [t.data_ptr() for t in grads], mast, [t.data_ptr() for t in m],
               [t.data_ptr() for t in v], *exps, sizes, _per_tensor(lr, n), _per_tensor(weight_decay, n))
    fields = [x for row in zip(*columns) for x in row]
    _lib.hylo_adamw_step(fields, n, pdt, gdt, bits, betas, eps, int(step), grad_scale, norm, max_norm, int(seed),
                         _lib.current_raw_stream(dev))
    increment_version(params)  # a backward through the values before the step raises, as after any in-place operation


class AdamW:
    """AdamW with its states. params: tensors, or dicts {"params": [...], "lr": ..., "weight_decay": ...} (groups).

    state_bits 32 or 8. bfloat16 parameters get fp32 masters unless masters=False. max_norm (optional)
    clips the global gradient norm of each step; ``last_norm`` is that norm (a device tensor). A step skipped for a norm
    that is not finite is counted in ``steps`` (the host does not wait to learn of it)."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.01,
                 state_bits: int = 32, masters: bool = True, max_norm: Optional[float] = None, seed: int = 0):
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        params = list(params)
        groups = params if params and isinstance(params[0], dict) else [{"params": params}]
        for g in groups:
            extra = set(g) - {"params", "lr", "weight_decay"}
            if extra:
                raise ValueError(f"a group of AdamW has its own lr and weight_decay only, not {', '.join(sorted(map(str, extra)))}")
        self.groups = [{"lr": lr, "weight_decay": weight_decay, **g, "params": list(g["params"])} for g in groups]
        self.betas, self.eps, self.max_norm, self.seed = tuple(betas), eps, max_norm, seed
        self.steps = 0
        self.last_norm: Optional[torch.Tensor] = None
        self.params = [p for g in self.groups for p in g["params"]]
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        if len({id(p) for p in self.params}) != len(self.params):
            raise ValueError("a parameter is given to AdamW twice")
        if any(p.dtype != self.params[0].dtype for p in self.params):
            raise ValueError("the parameters of one AdamW must share a dtype")
        def fresh(p):
            return State8.zeros_like(p) if state_bits == 8 else torch.zeros(p.shape, dtype=torch.float32, device=p.device)

        self.exp_avgs = [fresh(p) for p in self.params]
        self.exp_avg_sqs = [fresh(p) for p in self.params]
        self.masters = None
        if masters and self.params[0].dtype == torch.bfloat16:
            self.masters = [p.detach().float() for p in self.params]

    @torch.no_grad()
    def step(self, grads: Optional[Sequence[torch.Tensor]] = None, grad_scale: float = 1.0) -> None:
        """One step with `grads` (one per parameter, in order), or with the parameters' own .grad."""
        if grads is None:
            grads = [p.grad for p in self.params]
            if any(g is None for g in grads):
                raise ValueError("every parameter needs a gradient")
        self.last_norm = grad_norm(grads) if self.max_norm is not None else None
        lr = [g["lr"] for g in self.groups for _ in g["params"]]
        wd = [g["weight_decay"] for g in self.groups for _ in g["params"]]
        adamw_step([p.detach() for p in self.params], grads, self.exp_avgs, self.exp_avg_sqs, step=self.steps + 1, lr=lr,
                   betas=self.betas, eps=self.eps, weight_decay=wd, masters=self.masters, norm=self.last_norm,
                   max_norm=1.0 if self.max_norm is None else self.max_norm, grad_scale=grad_scale,
                   seed=self.seed + self.steps + 1)
        self.steps += 1

    def state_dict(self) -> dict:
        return {"steps": self.steps, "seed": self.seed, "exp_avgs": self.exp_avgs, "exp_avg_sqs": self.exp_avg_sqs,
                "masters": self.masters}

    def load_state_dict(self, state: dict) -> None:
        """Copies the states in (same parameters, state_bits and masters as when they were saved)."""
        def flat(d):
            out = []
            for x in (*d["exp_avgs"], *d["exp_avg_sqs"], *(d["masters"] or ())):
                out += x if isinstance(x, tuple) else [x]
            return out

        mine, theirs = flat(self.state_dict()), flat(state)
        if len(mine) != len(theirs) or any(a.shape != b.shape or a.dtype != b.dtype for a, b in zip(mine, theirs)):
            raise ValueError("the saved states do not match these parameters, state_bits and masters")
        for a, b in zip(mine, theirs):
            a.copy_(b)
        self.steps, self.seed = state["steps"], state["seed"]
