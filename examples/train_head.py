"""Trains a student's LM head and final hidden states against a teacher and given tokens, then scores the tokens.

One step: the distillation loss KL(teacher || student) plus the negative log-probability of the next tokens with
a small entropy bonus, both straight from hidden states and LM heads (the logits are never stored); then AdamW on
bfloat16 parameters with the gradient clipped on the device. With --layers the hidden states go through that many residual
layers first (RMS norm, matrix, sum in the next norm), whose matrices Muon steps. Afterwards the student's logits of a few
rows are scored once more with their five most probable alternatives.

    python examples/train_head.py --steps 20 --tokens 2048 --hidden 512 --vocab 32000 --state-bits 8 --layers 2
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from hybrid_upcycling_gb300 import AdamW, Muon, fused_hidden_state_kl, head_logprobs, rms_norm, token_logprobs  # noqa: E402


def student(h, gains, matrices):
    """Hidden states for the LM head: h through len(matrices) residual layers s <- s + norm(s) P^T, and a last norm."""
    if not gains:
        return h
    s, y = h, rms_norm(h, gains[0])
    for P, gain in zip(matrices, gains[1:]):
        y, s = rms_norm(y @ P.t(), gain, residual=s)
    return y


def train(steps: int = 20, tokens: int = 2048, hidden: int = 512, vocab: int = 32000, state_bits: int = 8,
          masters: bool = False, lr: float = 1e-2, seed: int = 0, device: str = "cuda", layers: int = 0):
    """(losses, mean log-probability before, after, alternatives of the first rows)."""
    gen = torch.Generator(device).manual_seed(seed)
    W_t = (torch.randn(vocab, 2 * hidden, generator=gen, device=device) * 0.02).bfloat16()
    h_t = torch.randn(tokens, 2 * hidden, generator=gen, device=device).bfloat16()
    target = torch.randint(0, vocab, (tokens,), generator=gen, device=device)
    target[::17] = -100  # positions without a next token
    W = (torch.randn(vocab, hidden, generator=gen, device=device) * 0.02).bfloat16().requires_grad_()
    h = torch.randn(tokens, hidden, generator=gen, device=device).bfloat16().requires_grad_()
    real = (target >= 0).sum()
    gains = [torch.ones(hidden, device=device).bfloat16().requires_grad_() for _ in range(layers + 1 if layers else 0)]
    matrices = [(torch.randn(hidden, hidden, generator=gen, device=device) * hidden ** -0.5).bfloat16().requires_grad_()
                for _ in range(layers)]

    def score():
        with torch.no_grad():
            return head_logprobs(student(h, gains, matrices), W, target)[0].sum() / real

    before = score()
    optimisers = [AdamW([{"params": [W], "weight_decay": 0.1}, {"params": [h, *gains], "weight_decay": 0.0}], lr=lr,
                        state_bits=state_bits, masters=masters, max_norm=1.0, seed=seed)]
    if layers:
        optimisers.append(Muon(matrices, lr=lr, weight_decay=0.1, masters=masters, max_norm=1.0, adjust="rms", seed=seed))
    losses = []
    for _ in range(steps):
        y = student(h, gains, matrices)
        kl, _ = fused_hidden_state_kl(y, W, h_t, W_t)
        logp, entropy = head_logprobs(y, W, target)
        loss = kl - logp.sum() / real - 0.01 * entropy.mean()
        for p in (W, h, *gains, *matrices):
            p.grad = None
        loss.backward()
        for opt in optimisers:
            opt.step()
        losses.append(loss.detach())
    after = score()
    with torch.no_grad():
        top = token_logprobs(student(h, gains, matrices)[:4] @ W.t(), target[:4], top_k=5)
    return torch.stack(losses).tolist(), before.item(), after.item(), top


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--vocab", type=int, default=32000)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    ap.add_argument("--layers", type=int, default=0)
    ap.add_argument("--masters", action="store_true", help="fp32 copies of the parameters")
    a = ap.parse_args()
    losses, before, after, top = train(a.steps, a.tokens, a.hidden, a.vocab, a.state_bits, a.masters, layers=a.layers)
    print("loss %.4f -> %.4f, mean log-probability of the tokens %.3f -> %.3f" % (losses[0], losses[-1], before, after))
    for r in range(top.top_tokens.shape[0]):
        print("row %d: entropy %.3f, alternatives %s" % (r, top.entropy[r].item(), ", ".join(
            "%d (%.2f)" % x for x in zip(top.top_tokens[r].tolist(), top.top_logprobs[r].tolist()))))


if __name__ == "__main__":
    main()
