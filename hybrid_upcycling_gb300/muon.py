"""Orthogonalised updates: ``orthogonalize`` (Newton-Schulz steps on the tensor cores), ``muon_step`` and ``Muon``.

Muon steps matrices: momentum, the update's orthogonal factor, weight decay. ``AdamW`` is for everything else (gains, biases,
embeddings, the LM head). include/hylo_ops.h has the formulas. PyTorch only allocates memory; the calls run on the current
stream and never wait for the host.
"""
from __future__ import annotations

import math
import struct
from typing import Iterable, List, Optional, Sequence, Tuple, Union

import torch
from torch.autograd.forward_ad import unpack_dual
from torch.autograd.graph import increment_version

from . import _lib
from .optim import _check_list, _per_tensor, grad_norm

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
Coefficients = Union[Tuple[float, float, float], Sequence[Tuple[float, float, float]]]


def _coefficients(coefficients: Coefficients, steps: int) -> List[float]:
    """Three numbers for each step, one after another: one triple serves all steps."""
    rows = list(coefficients)
    if len(rows) == 3 and not any(isinstance(x, (tuple, list)) for x in rows):
        rows = [rows] * int(steps)
    if len(rows) != steps or any(not isinstance(r, (tuple, list)) or len(r) != 3 for r in rows):
        raise ValueError("coefficients are three numbers, or as many triples as there are steps")
    return [float(x) for r in rows for x in r]


def _workspace(n: int, device) -> torch.Tensor:
    if n == 0:
        raise ValueError("invalid sizes: sides up to 2^20, the shorter up to 16384")
    return torch.empty(n, dtype=torch.uint8, device=device)  # from the caching allocator of the current stream


def _upright(x: torch.Tensor) -> Tuple[torch.Tensor, bool]:
    """x [..., m, n] with unit column stride and rows that do not overlap, or its transpose if that has them."""
    if x.stride(-1) == 1 or x.shape[-1] == 1:
        flipped = False
    elif x.stride(-2) == 1 or x.shape[-2] == 1:
        x, flipped = x.transpose(-1, -2), True
    else:
        return x.contiguous(), False
    if (x.shape[-1] > 1 and x.stride(-1) != 1) or (x.shape[-2] > 1 and x.stride(-2) < x.shape[-1]):
        x = x.contiguous()
    return x, flipped


class _Result(torch.autograd.Function):
    """A result as a function of its matrix, of which no derivative is implemented."""
    @staticmethod
    def forward(ctx, result, matrix):
        ctx.mark_dirty(result)  # the tensor itself, not a view: it may be written in place
        return result

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("orthogonalize is not differentiable: detach its matrices or its results")


def orthogonalize(matrices: Union[torch.Tensor, Iterable[torch.Tensor]], steps: int = 5,
                  coefficients: Coefficients = COEFFICIENTS, eps: float = 1e-7, dtype: torch.dtype = torch.bfloat16):
    """The matrices with their singular values brought near 1, by ``steps`` Newton-Schulz steps from X = M / (|M| + eps):
    X <- a X + (b A + c A^2) X with A = X X^T.

    matrices: a list of tensors [..., m, n], all float32, bfloat16 or float16, leading dimensions being a batch of matrices, or
    one such tensor. Rows or columns with unit stride are read in place. Returns contiguous tensors (or one) of ``dtype``,
    bfloat16 or float16: the products take fp16 numbers, 1e-3 to 2e-3 of the result's norm (up to 4e-3 for a single row).
    coefficients: (a, b, c), or one triple for each step. Not differentiable: a backward through a result raises, and
    forward-mode tensors are refused."""
    single = isinstance(matrices, torch.Tensor)
    tensors = [matrices] if single else list(matrices)
    if dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("dtype must be bfloat16 or float16")
    k = _coefficients(coefficients, steps)
    if any(unpack_dual(x).tangent is not None for x in tensors):
        raise NotImplementedError("orthogonalize has no forward-mode derivatives")
    for x in tensors:
        if x.dim() < 2 or x.dtype not in _lib.DTYPES or x.dtype != tensors[0].dtype:
            raise ValueError("matrices must be [..., m, n], all float32, all bfloat16 or all float16")
        if not x.is_cuda or x.get_device() != torch.cuda.current_device():
            raise ValueError("matrices must be on the current CUDA device")
    out: List[torch.Tensor] = []
    fields, kept, count = [], [], 0
    for x in tensors:
        y, flipped = _upright(x.detach())
        r = torch.empty(y.shape, dtype=dtype, device=x.device)
        out.append(r.transpose(-1, -2) if flipped else r)
        if r.numel() == 0:
            continue
        kept.append(y)
        rows, cols = y.shape[-2:]
        ld = y.stride(-2) if rows > 1 else cols
        batch = y.reshape(-1, rows, cols) if y.dim() > 3 else y  # a copy where the batch has no one stride
        if batch.dim() == 3:
            if rows > 1:
                ld = batch.stride(1)
            kept.append(batch)
            step, size = batch.stride(0) * y.element_size(), rows * cols * r.element_size()
            for i in range(batch.shape[0]):
                fields += (batch.data_ptr() + i * step, r.data_ptr() + i * size, rows, cols, ld)
            count += batch.shape[0]
        else:
            fields += (y.data_ptr(), r.data_ptr(), rows, cols, ld)
            count += 1
    if count:
        device = tensors[0].device
        table = struct.pack("=" + _lib.ORTH_MATRIX * count, *fields)
        ws = _workspace(_lib.hylo_orthogonalize_workspace_bytes(table, count), device)
        _lib.hylo_orthogonalize(table, count, tensors[0].dtype, dtype, k, float(eps), ws, _lib.current_raw_stream(device.index))
    out = [r.contiguous() for r in out]  # a copy of what was read by its columns
    if torch.is_grad_enabled():
        out = [_Result.apply(r, x) if x.requires_grad else r for r, x in zip(out, tensors)]
    return out[0] if single else out


def _scale(adjust: Optional[str], rows: int, cols: int) -> float:
    if adjust == "shape":
        return math.sqrt(max(1.0, rows / max(1, cols)))
    if adjust == "rms":
        return 0.2 * math.sqrt(max(rows, cols))
    if adjust is None:
        return 1.0
    raise ValueError('adjust must be "shape", "rms" or None')


def muon_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], momenta: Sequence[torch.Tensor], *, lr,
              momentum: float = 0.95, nesterov: bool = True, weight_decay=0.0, steps: int = 5,
              coefficients: Coefficients = COEFFICIENTS, eps: float = 1e-7, adjust: Optional[str] = "shape",
              masters: Optional[Sequence[torch.Tensor]] = None, norm: Optional[torch.Tensor] = None,
              max_norm: float = 1.0, grad_scale: float = 1.0, seed: int = 0) -> None:
    """One Muon step, in place, over lists of matrices [..., m, n] (leading dimensions: a batch of matrices). Tensors that are
    written may not overlap.

        momentum buffer <- momentum buffer + (1 - momentum) grad;  update: that, or with ``nesterov`` one more such step
        param <- param (1 - lr weight_decay) - lr scale orthogonalize(update)

    params, grads, masters, norm, max_norm, grad_scale and seed as in ``adamw_step``; momenta: float32 tensors. lr and
    weight_decay: numbers, or one per tensor. adjust: scale = sqrt(max(1, m / n)) ("shape"), 0.2 sqrt(max(m, n)), which gives
    the update the size of an AdamW step ("rms"), or 1 (None). steps, coefficients, eps as in ``orthogonalize``. A step
    cannot be captured into a CUDA graph: lr and seed are host values, which every replay would repeat."""
    params, grads, momenta = list(params), list(grads), list(momenta)
    n = len(params)
    if not (len(grads) == len(momenta) == n and (masters is None or len(masters) == n)):
        raise ValueError("params, grads, momenta and masters must have the same length")
    k = _coefficients(coefficients, steps)
    _scale(adjust, 1, 1)
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
    for i, p in enumerate(params):
        if p.dim() < 2:
            raise ValueError(f"params[{i}] must be a matrix or a batch of matrices")
    for name, tensors, dtype in (("params", params, pdt), ("grads", grads, gdt), ("momenta", momenta, torch.float32),
                                 ("masters", masters or (), torch.float32)):
        _check_list(name, tensors, (dtype,), dev)
        for i, t in enumerate(tensors):
            if t.shape != params[i].shape:
                raise ValueError(f"{name}[{i}] must have the shape of params[{i}]")
    lr, weight_decay = _per_tensor(lr, n), _per_tensor(weight_decay, n)
    fields, count = [], 0
    for i, p in enumerate(params):
        rows, cols = p.shape[-2:]
        arrays = (p, grads[i], None if masters is None else masters[i], momenta[i])
        scale, size = _scale(adjust, rows, cols), rows * cols
        for b in range(p.numel() // size if size else 0):
            fields += [0 if t is None else t.data_ptr() + b * size * t.element_size() for t in arrays]
            fields += (rows, cols, lr[i], weight_decay[i], scale)
            count += 1
    if count == 0:
        return
    table = struct.pack("=" + _lib.MUON_TENSOR * count, *fields)
    ws = _workspace(_lib.hylo_muon_workspace_bytes(table, count), params[0].device)
    _lib.hylo_muon_step(table, count, pdt, gdt, float(momentum), bool(nesterov), k, float(eps), float(grad_scale), norm,
                        float(max_norm), int(seed), ws, _lib.current_raw_stream(dev))
    increment_version(params)  # a backward through the values before the step raises, as after any in-place operation


class Muon:
    """Muon with its momenta. params: matrices (or batches of them), or dicts {"params": [...], "lr": ..., "weight_decay": ...}
    (groups); everything that is not a matrix belongs to ``AdamW``.

    bfloat16 parameters get fp32 masters unless masters=False. max_norm (optional) clips the global gradient norm of each step,
    which counts in the momentum; ``last_norm`` is that norm (a device tensor). A step skipped for a norm that is not finite is
    counted in ``steps`` (the host does not wait to learn of it)."""

    def __init__(self, params, lr: float = 0.02, momentum: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0,
                 ns_steps: int = 5, coefficients: Coefficients = COEFFICIENTS, eps: float = 1e-7,
                 adjust: Optional[str] = "shape", masters: bool = True, max_norm: Optional[float] = None, seed: int = 0):
        _coefficients(coefficients, ns_steps)
        _scale(adjust, 1, 1)
        params = list(params)
        groups = params if params and isinstance(params[0], dict) else [{"params": params}]
        for g in groups:
            extra = set(g) - {"params", "lr", "weight_decay"}
            if extra:
                raise ValueError(f"a group of Muon has its own lr and weight_decay only, not {', '.join(sorted(map(str, extra)))}")
        self.groups = [{"lr": lr, "weight_decay": weight_decay, **g, "params": list(g["params"])} for g in groups]
        self.momentum, self.nesterov, self.ns_steps, self.coefficients = momentum, nesterov, ns_steps, coefficients
        self.eps, self.adjust, self.max_norm, self.seed = eps, adjust, max_norm, seed
        self.steps = 0
        self.last_norm: Optional[torch.Tensor] = None
        self.params = [p for g in self.groups for p in g["params"]]
        if not self.params:
            raise ValueError("Muon needs at least one parameter")
        if len({id(p) for p in self.params}) != len(self.params):
            raise ValueError("a parameter is given to Muon twice")
        if any(p.dtype != self.params[0].dtype for p in self.params):
            raise ValueError("the parameters of one Muon must share a dtype")
        if any(p.dim() < 2 for p in self.params):
            raise ValueError("Muon steps matrices: give vectors and numbers to AdamW")
        self.momenta = [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in self.params]
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
        muon_step([p.detach() for p in self.params], grads, self.momenta, lr=lr, momentum=self.momentum,
                  nesterov=self.nesterov, weight_decay=wd, steps=self.ns_steps, coefficients=self.coefficients, eps=self.eps,
                  adjust=self.adjust, masters=self.masters, norm=self.last_norm,
                  max_norm=1.0 if self.max_norm is None else self.max_norm, grad_scale=grad_scale,
                  seed=self.seed + self.steps + 1)
        self.steps += 1

    def state_dict(self) -> dict:
        return {"steps": self.steps, "seed": self.seed, "momenta": self.momenta, "masters": self.masters}

    def load_state_dict(self, state: dict) -> None:
        """Copies the states in (same parameters and masters as when they were saved)."""
        def flat(d):
            return [*d["momenta"], *(d["masters"] or ())]

        mine, theirs = flat(self.state_dict()), flat(state)
        if len(mine) != len(theirs) or any(a.shape != b.shape or a.dtype != b.dtype for a, b in zip(mine, theirs)):
            raise ValueError("the saved states do not match these parameters and masters")
        for a, b in zip(mine, theirs):
            a.copy_(b)
        self.steps, self.seed = state["steps"], state["seed"]
