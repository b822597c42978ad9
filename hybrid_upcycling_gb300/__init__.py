"""GB300-native (sm_103a) fused hidden-state KL distillation loss of HyLo's Stage II.

The compute lives in libhylo_kl.so (hand-written tcgen05/TMA kernels behind the C ABI of
include/hylo_kl.h and include/hylo_ops.h). ``_lib`` binds that ABI one-to-one; ``kl`` wraps the three
losses as PyTorch autograd functions, ``logprobs`` the log-probabilities of given tokens; ``optim`` is the
AdamW step that applies the gradients; ``synthetic`` draws the seeded benchmark inputs.
"""
from . import synthetic  # noqa: F401

__all__ = ["synthetic", "fused_hidden_state_kl", "fused_logits_kl", "ild_loss", "token_logprobs", "TokenLogprobs",
           "head_logprobs", "grad_norm", "adamw_step", "AdamW", "State8"]

_LAZY = {"token_logprobs": "logprobs", "TokenLogprobs": "logprobs", "head_logprobs": "logprobs", "grad_norm": "optim",
         "adamw_step": "optim", "AdamW": "optim", "State8": "optim"}


def __getattr__(name):
    if name not in _LAZY:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from importlib import import_module
    globals()[name] = value = getattr(import_module("." + _LAZY[name], __name__), name)
    return value


def fused_hidden_state_kl(*args, **kwargs):
    from .kl import fused_hidden_state_kl as f
    return f(*args, **kwargs)


def fused_logits_kl(*args, **kwargs):
    from .kl import fused_logits_kl as f
    return f(*args, **kwargs)


def ild_loss(*args, **kwargs):
    from .kl import ild_loss as f
    return f(*args, **kwargs)
